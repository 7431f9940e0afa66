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
__device__ __forceinline__ void load_row(const bf16* src, float* x) {  // D values, 16 bytes at a time
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(src) + i);
    const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[8 * i + 2 * e] = bf16_lo(a[e]);
      x[8 * i + 2 * e + 1] = bf16_hi(a[e]);
    }
  }
}

// value c of cache row `row`
template <int D, int KV>
__device__ __forceinline__ float kv_at(const AttendParams& p, bool value, int64_t row, int c) {
  if constexpr (KV == kKvPagedE4m3) {
    const uint8_t code = static_cast<const uint8_t*>(value ? p.pages.V : p.pages.K)[row * D + c];
    return bf16_lo(e4m3x2_to_bf16x2(code)) * (value ? p.pages.vs : p.pages.ks)[row];
  } else {
    const bf16* x = KV == kKvPlain ? (value ? p.V : p.K) : static_cast<const bf16*>(value ? p.pages.V : p.pages.K);
    return __bfloat162float(x[row * D + c]);
  }
}

template <int D, int KV>
__global__ void __launch_bounds__(32 * kRowWarps) attend_rows_kernel(const AttendParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t row = int64_t(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  if (row >= int64_t(p.B) * p.Hq * p.N) return;
  const int t = int(row % p.N), h = int((row / p.N) % p.Hq), b = int(row / p.N / p.Hq);
  const int hk = h / (p.Hq / p.Hkv);
  int n = p.N, pos = t;
  if constexpr (KV != kKvPlain) {
    n = kv_len_of(p.pages, b);
    const int nq = q_len_of(p.pages, b, p.N);
    if (t >= nq) return;
    pos = n - nq + t;
  }
  __shared__ float qs[kRowWarps][D];
  float* q = qs[threadIdx.x >> 5];
  for (int c = lane; c < D; c += 32) q[c] = __bfloat162float(p.Q[row * D + c]) * p.scale;
  __syncwarp();
  float m = -INFINITY, l = 0.f, o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
  const int hi = max(0, min(n, pos + p.win.right + 1)), lo = max(0, pos - p.win.left);
  for (int j0 = 0; j0 < hi; j0 += 32) {
    if (j0 >= p.win.sinks && j0 + 32 <= lo) continue;
    const int j = j0 + lane;
    bool see = j < hi && p.win.sees(pos, j);
    int64_t at = (int64_t(b) * p.Hkv + hk) * p.N + j;
    if constexpr (KV != kKvPlain) {
      const int page = see ? page_of(p.pages, b, j) : -1;
      see = page >= 0;
      at = ((int64_t(page) * p.Hkv + hk) << p.pages.log_page) + (j & ((1 << p.pages.log_page) - 1));
    }
    float s = -INFINITY;
    if (see) {
      s = 0.f;
      for (int c = 0; c < D; ++c) s = fmaf(q[c], kv_at<D, KV>(p, false, at, c), s);
    }
    float mx = s;
    for (int off = 16; off; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, off));
    mx = fmaxf(m, mx);
    if (mx == -INFINITY) mx = 0.f;
    const float f = __expf(m - mx), w = see ? __expf(s - mx) : 0.f;
    m = mx;
    l *= f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] *= f;
    const unsigned any = __ballot_sync(~0u, see);
    for (unsigned k = any; k; k &= k - 1) {
      const int from = __ffs(k) - 1;
      const float wk = __shfl_sync(~0u, w, from);
      const int64_t r = __shfl_sync(~0u, at, from);
      l += wk;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) o[i] = fmaf(wk, kv_at<D, KV>(p, true, r, i * 32 + lane), o[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < D / 32; ++i) p.O[row * D + i * 32 + lane] = __float2bfloat16(l > 0.f ? o[i] / l : o[i]);
  if (lane == 0 && p.lse) p.lse[row] = l > 0.f ? m + logf(l) : (l == 0.f ? -INFINITY : l);
}

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
