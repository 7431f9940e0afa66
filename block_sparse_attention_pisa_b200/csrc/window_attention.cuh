// Attention with a token-exact window and first tokens that stay visible, over keys laid out
// plainly ([B, Hkv, N, D]) or in pages, and its gradient. One warp per query row (forward,
// dQ) or per key row (dK, dV); the keys of a row are taken 32 at a time, one per lane.
//
//   s_j = scale q.k_j on the visible keys, lse = log sum exp s, o = sum exp(s - lse) v
//   delta = do.o, ds_j = p_j (do.v_j - delta), dq = scale sum ds_j k_j,
//   dk_j = scale sum ds_j q, dv_j = sum p_j do   (sums over rows and the heads of a group)
#pragma once

#include "window.cuh"

namespace pisa {

struct AttendParams {
  const bf16* Q;
  const bf16* K;  // plain keys and values; or `pages`
  const bf16* V;
  Pages pages;
  bf16* O;
  float* lse;
  int B, Hq, Hkv, N;
  Window win;
  float scale;
  // gradient
  const bf16* dO;
  bf16 *dQ, *dK, *dV;
  float* delta;
};

constexpr int kRowWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kRowWarps) attend_delta_kernel(const AttendParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (row >= int64_t(p.B) * p.Hq * p.N) return;
  float s = 0.f;
  for (int c = lane; c < D; c += 32) s += __bfloat162float(p.dO[row * D + c]) * __bfloat162float(p.O[row * D + c]);
  for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(~0u, s, off);
  if (lane == 0) p.delta[row] = s;
}

// dQ of one row: keys one at a time, lanes over the dimensions
template <int D>
__global__ void __launch_bounds__(32 * kRowWarps) attend_dq_kernel(const AttendParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (row >= int64_t(p.B) * p.Hq * p.N) return;
  const int t = int(row % p.N), h = int((row / p.N) % p.Hq), b = int(row / p.N / p.Hq);
  const int64_t kv0 = (int64_t(b) * p.Hkv + h / (p.Hq / p.Hkv)) * p.N;
  float q[D / 32], g[D / 32], dq[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    q[i] = __bfloat162float(p.Q[row * D + i * 32 + lane]) * p.scale;
    g[i] = __bfloat162float(p.dO[row * D + i * 32 + lane]);
    dq[i] = 0.f;
  }
  const float lse = p.lse[row], delta = p.delta[row];
  for (int j = 0; j < p.N; ++j) {
    if (!p.win.sees(t, j)) continue;
    float s = 0.f, w = 0.f, k[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      k[i] = __bfloat162float(p.K[(kv0 + j) * D + i * 32 + lane]);
      s = fmaf(q[i], k[i], s);
      w = fmaf(g[i], __bfloat162float(p.V[(kv0 + j) * D + i * 32 + lane]), w);
    }
    for (int off = 16; off; off >>= 1) {
      s += __shfl_xor_sync(~0u, s, off);
      w += __shfl_xor_sync(~0u, w, off);
    }
    const float ds = __expf(s - lse) * (w - delta);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) dq[i] = fmaf(ds, k[i], dq[i]);
  }
#pragma unroll
  for (int i = 0; i < D / 32; ++i) p.dQ[row * D + i * 32 + lane] = __float2bfloat16(dq[i] * p.scale);
}

// dK, dV of one key row: the rows of the group's heads that see it
template <int D>
__global__ void __launch_bounds__(32 * kRowWarps) attend_dkv_kernel(const AttendParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t key = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (key >= int64_t(p.B) * p.Hkv * p.N) return;
  const int j = int(key % p.N), hk = int((key / p.N) % p.Hkv), b = int(key / p.N / p.Hkv);
  const int G = p.Hq / p.Hkv;
  float k[D / 32], v[D / 32], dk[D / 32], dv[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    k[i] = __bfloat162float(p.K[key * D + i * 32 + lane]);
    v[i] = __bfloat162float(p.V[key * D + i * 32 + lane]);
    dk[i] = dv[i] = 0.f;
  }
  for (int h = hk * G; h < hk * G + G; ++h)
    for (int t = 0; t < p.N; ++t) {
      if (!p.win.sees(t, j)) continue;
      const int64_t row = (int64_t(b) * p.Hq + h) * p.N + t;
      float s = 0.f, w = 0.f, q[D / 32], g[D / 32];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        q[i] = __bfloat162float(p.Q[row * D + i * 32 + lane]);
        g[i] = __bfloat162float(p.dO[row * D + i * 32 + lane]);
        s = fmaf(q[i] * p.scale, k[i], s);
        w = fmaf(g[i], v[i], w);
      }
      for (int off = 16; off; off >>= 1) {
        s += __shfl_xor_sync(~0u, s, off);
        w += __shfl_xor_sync(~0u, w, off);
      }
      const float pj = __expf(s - p.lse[row]), ds = pj * (w - p.delta[row]) * p.scale;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        dk[i] = fmaf(ds, q[i], dk[i]);
        dv[i] = fmaf(pj, g[i], dv[i]);
      }
    }
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    p.dK[key * D + i * 32 + lane] = __float2bfloat16(dk[i]);
    p.dV[key * D + i * 32 + lane] = __float2bfloat16(dv[i]);
  }
}

}  // namespace pisa
