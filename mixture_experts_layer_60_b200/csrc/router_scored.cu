// Scored router (moe_route_scored): softmax or sigmoid scores of u E^T, biased
// and group-limited top-K, gates, load.
//
// Logits come as S partial sums over slices of d, [S][T][ld]:
//   float64 (router_logits64_kernel): float32 inputs, and few bf16 tokens;
//     every key is then the definition's and nothing has to be redone.
// A warp per token joins the slices and routes (router_select.cuh).
#include "launch.h"
#include "router_select.cuh"

namespace moe {

namespace {

// ---------------------------------------------------------------- float64 logits
// P[s][t][i] = sum over slice s of d of u[t,k] E[i,k], float64 products and
// sums.  A 32-token x 32-expert tile per block of 256 threads (2 x 2 outputs a
// thread), 32 columns of both operands staged in shared memory as float64.
// Bound by the float64 rate (64 FMA per SM and cycle) and shared memory.
constexpr int kT64 = 32;

template <typename Tin>
__global__ void __launch_bounds__(256) router_logits64_kernel(
    const Tin* __restrict__ u, const Tin* __restrict__ E, int T, int d, int N, int S, int ld,
    double* __restrict__ P, int32_t* __restrict__ counts) {
  __shared__ double su[kT64][kT64 + 1], se[kT64][kT64 + 1];
  const int tid = threadIdx.x;
  const int t0 = blockIdx.x * kT64, e0 = blockIdx.y * kT64, sl = blockIdx.z;
  if (blockIdx.x == 0 && blockIdx.y == 0 && sl == 0)
    for (int i = tid; i < N; i += 256) counts[i] = 0;
  const int nc = d / kT64;                                // d % 64 == 0
  const int c0 = (int)((long long)sl * nc / S), c1 = (int)((long long)(sl + 1) * nc / S);
  const int tx = tid & 15, ty = tid >> 4;                 // experts tx, tx+16; tokens ty, ty+16
  double a00 = 0, a01 = 0, a10 = 0, a11 = 0;
  for (int c = c0; c < c1; ++c) {
    for (int i = tid; i < kT64 * kT64; i += 256) {
      const int r = i >> 5, k = i & 31;
      su[r][k] = t0 + r < T ? (double)IO<Tin>::ld(u + (size_t)(t0 + r) * d + c * kT64 + k) : 0.0;
      se[r][k] = e0 + r < N ? (double)IO<Tin>::ld(E + (size_t)(e0 + r) * d + c * kT64 + k) : 0.0;
    }
    __syncthreads();
#pragma unroll 8
    for (int k = 0; k < kT64; ++k) {
      const double x0 = su[ty][k], x1 = su[ty + 16][k], y0 = se[tx][k], y1 = se[tx + 16][k];
      a00 = fma(x0, y0, a00);
      a01 = fma(x0, y1, a01);
      a10 = fma(x1, y0, a10);
      a11 = fma(x1, y1, a11);
    }
    __syncthreads();
  }
  double* out = P + (size_t)sl * T * ld;
  const double v[2][2] = {{a00, a01}, {a10, a11}};
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int t = t0 + ty + 16 * i, e = e0 + tx + 16 * j;
      if (t < T && e < N) out[(size_t)t * ld + e] = v[i][j];
    }
}

// ---------------------------------------------------------------- selection
// A warp per token; the block's load histogram in shared memory, then added to
// counts (whole numbers: the order of the additions does not matter).
template <int V>
__global__ void __launch_bounds__(256) router_select64_kernel(
    const double* __restrict__ P, int S, int ld, const float* __restrict__ bias, int T,
    SelectRule r, int32_t* __restrict__ idx, float* __restrict__ gate,
    int32_t* __restrict__ counts, float* __restrict__ logits) {
  extern __shared__ int hist[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wpb = blockDim.x >> 5;
  const int N = r.N_r;
  float* wk = reinterpret_cast<float*>(hist + N) + (size_t)warp * N;
  for (int i = threadIdx.x; i < N; i += blockDim.x) hist[i] = 0;
  __syncthreads();
  for (int t = blockIdx.x * wpb + warp; t < T; t += gridDim.x * wpb) {
    const auto getx = [&](int e) {
      double v = 0.0;
      for (int s = 0; s < S; ++s) v += P[((size_t)s * T + t) * ld + e];
      return v;
    };
    double x[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = j * 32 + lane;
      x[j] = e < N ? getx(e) : 0.0;
      if (logits && e < N) logits[(size_t)t * N + e] = (float)x[j];
    }
    select_token<V, double>(x, getx, bias, r, 0.f, wk, idx + (size_t)t * r.K,
                            gate + (size_t)t * r.K);
    for (int k = lane; k < r.K; k += 32) atomicAdd(&hist[idx[(size_t)t * r.K + k]], 1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < N; i += blockDim.x)
    if (hist[i]) atomicAdd(&counts[i], hist[i]);
}

// Slices of d for the float64 logits: enough blocks for two per SM, at most
// kMaxSlices64, each slice at least 128 columns.
constexpr int kMaxSlices64 = 16;
int slices64(int T, int d, int N) {
  const long long tiles = (long long)((T + kT64 - 1) / kT64) * ((N + kT64 - 1) / kT64);
  long long S = (2LL * 148 + tiles - 1) / tiles;
  if (S > d / 128) S = d / 128;
  if (S > kMaxSlices64) S = kMaxSlices64;
  return S < 1 ? 1 : (int)S;
}

int dispatch_v(int N) {
  const int V = (N + 31) / 32;
  return V <= 1 ? 1 : V <= 2 ? 2 : V <= 4 ? 4 : V <= 8 ? 8 : V <= 16 ? 16 : 32;
}

}  // namespace

size_t route_scored_ws_bytes(int T, int d, int N_r) {
  return align_up((size_t)slices64(T, d, N_r) * T * N_r * sizeof(double), 256);
}

moe_status launch_route_scored(const void* u, const void* E, moe_dtype dt, const float* b, int T,
                               int d, int N_r, int K, int score, int n_groups, int topk_groups,
                               int group_top, int renorm, float gate_scale, int32_t* idx,
                               float* gate, int32_t* counts, float* logits, void* ws,
                               cudaStream_t s) {
  const SelectRule r{N_r, K, score, n_groups, topk_groups, group_top, renorm, gate_scale};
  double* P = static_cast<double*>(ws);
  const int S = slices64(T, d, N_r);
  const dim3 grid((T + kT64 - 1) / kT64, (N_r + kT64 - 1) / kT64, S);
  if (dt == MOE_F32)
    router_logits64_kernel<float><<<grid, 256, 0, s>>>(static_cast<const float*>(u),
                                                       static_cast<const float*>(E), T, d, N_r, S,
                                                       N_r, P, counts);
  else
    router_logits64_kernel<__nv_bfloat16><<<grid, 256, 0, s>>>(
        static_cast<const __nv_bfloat16*>(u), static_cast<const __nv_bfloat16*>(E), T, d, N_r, S,
        N_r, P, counts);
  moe_status st = cuda_check(cudaGetLastError(), "router_logits64 launch");
  if (st != MOE_OK) return st;
  const int wpb = 4;
  int blocks = (T + wpb - 1) / wpb;
  if (blocks > 16 * sm_count()) blocks = 16 * sm_count();
  const size_t smem = (size_t)N_r * sizeof(int) * (1 + wpb);
#define MOE_SELECT64(v)                                                                      \
  case v:                                                                                    \
    router_select64_kernel<v><<<blocks, wpb * 32, smem, s>>>(P, S, N_r, b, T, r, idx, gate,  \
                                                             counts, logits);                \
    break;
  switch (dispatch_v(N_r)) {
    MOE_SELECT64(1) MOE_SELECT64(2) MOE_SELECT64(4) MOE_SELECT64(8) MOE_SELECT64(16)
    MOE_SELECT64(32)
  }
#undef MOE_SELECT64
  return cuda_check(cudaGetLastError(), "router_select64 launch");
}

}  // namespace moe
