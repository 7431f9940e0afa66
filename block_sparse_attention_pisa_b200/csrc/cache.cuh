// Paged key/value cache: rows are quantised as they are written, and read back.
//
// A row is one token of one key head (d values). In 8 bits it is held as e4m3 codes with one
// fp32 scale: scale = max(amax|x| / 448, 2^-126), code = e4m3(x / scale) (IEEE division, round
// to nearest even, so the codes are those of the formula), and read back as
// bf16(code * scale). The bits of |x| grow with |x| and a NaN's lie above infinity's, so the
// maximum is taken over the bits: a row with a NaN or an infinity gets the scale NaN, and the
// whole row reads back as NaN.
//
// Both kernels are bound by memory: each row of x is read once and its codes written once
// (or the reverse), 16 bytes of x per thread and row, a row per D/8 neighbouring threads; the
// lengths, the page table and the scales are small beside that.
#pragma once

#include "window.cuh"

namespace pisa {

constexpr int kCacheThreads = 256;
constexpr int kCacheRows = 4;  // rows in flight per thread

struct CacheParams {
  Pages pages;
  void* cK;
  void* cV;
  float* ks;
  float* vs;
  const bf16* K;
  const bf16* V;
  bf16* oK;
  bf16* oV;
  int Hkv, N;
  int64_t rows;  // B * Hkv * N
};

// cache row of token t of (b, h), or -1
__device__ __forceinline__ int64_t cache_row(const CacheParams& p, int b, int h, int pos) {
  const int at = page_of(p.pages, b, pos);
  return at < 0 ? -1 : ((int64_t(at) * p.Hkv + h) << p.pages.log_page) + (pos & ((1 << p.pages.log_page) - 1));
}

// 8 bf16 (one 16-byte load) -> the row's scale and 8 codes
template <int D>
__device__ __forceinline__ uint2 quantise8(const uint4& x, float& scale) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
#pragma unroll
  for (int off = 1; off < D / 8; off <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
  if (top >= 0x7f80u) top = 0x7fc0u;  // an infinity or a NaN: NaN for the row
  scale = __fdiv_rn(__uint_as_float(top << 16), 448.f);
  if (scale < 1.17549435e-38f) scale = 1.17549435e-38f;  // a NaN stays one
  uint32_t c[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 f = make_float4(__fdiv_rn(bf16_lo(w[2 * i]), scale), __fdiv_rn(bf16_hi(w[2 * i]), scale),
                                 __fdiv_rn(bf16_lo(w[2 * i + 1]), scale), __fdiv_rn(bf16_hi(w[2 * i + 1]), scale));
    c[i] = uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(f.x, f.y), __NV_SATFINITE, __NV_E4M3)) |
           uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(f.z, f.w), __NV_SATFINITE, __NV_E4M3)) << 16;
  }
  return make_uint2(c[0], c[1]);
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kCacheThreads) cache_write_kernel(const CacheParams p) {
  constexpr int LPR = D / 8;  // threads per row
  const int part = threadIdx.x % LPR;
  const int64_t step = int64_t(gridDim.x) * (kCacheThreads / LPR);
  const int64_t first = int64_t(blockIdx.x) * (kCacheThreads / LPR) + threadIdx.x / LPR;
  // every thread of a warp takes the same number of rounds (the shuffles need all lanes)
  for (int64_t r0 = first - threadIdx.x / LPR; r0 < p.rows; r0 += step * kCacheRows) {
    uint4 k[kCacheRows], v[kCacheRows];
    int64_t to[kCacheRows];
#pragma unroll
    for (int i = 0; i < kCacheRows; ++i) {
      const int64_t r = r0 + threadIdx.x / LPR + i * step;
      to[i] = -1;
      k[i] = v[i] = make_uint4(0, 0, 0, 0);
      if (r < p.rows) {
        const uint32_t bh = uint32_t(r) / uint32_t(p.N), t = uint32_t(r) % uint32_t(p.N);
        const int b = bh / p.Hkv, h = bh % p.Hkv;
        const int n = q_len_of(p.pages, b, p.N), pos = kv_len_of(p.pages, b) - n + int(t);
        if (int(t) < n && pos >= 0) {
          to[i] = cache_row(p, b, h, pos);
          k[i] = ldg_stream_v4(p.K + r * D + part * 8);
          v[i] = ldg_stream_v4(p.V + r * D + part * 8);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kCacheRows; ++i) {
      if constexpr (E4M3) {
        float ks, vs;
        const uint2 kc = quantise8<D>(k[i], ks), vc = quantise8<D>(v[i], vs);
        if (to[i] >= 0) {
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.cK) + to[i] * D + part * 8) = kc;
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.cV) + to[i] * D + part * 8) = vc;
          if (part == 0) {
            p.ks[to[i]] = ks;
            p.vs[to[i]] = vs;
          }
        }
      } else if (to[i] >= 0) {
        *reinterpret_cast<uint4*>(static_cast<bf16*>(p.cK) + to[i] * D + part * 8) = k[i];
        *reinterpret_cast<uint4*>(static_cast<bf16*>(p.cV) + to[i] * D + part * 8) = v[i];
      }
    }
  }
}

// 8 codes and their scale -> 8 bf16
__device__ __forceinline__ uint4 restore8(const uint2& c, float scale) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t two = e4m3x2_to_bf16x2(i < 2 ? c.x >> (16 * i) : c.y >> (16 * (i - 2)));
    w[i] = pack_bf16x2(bf16_lo(two) * scale, bf16_hi(two) * scale);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kCacheThreads) cache_read_kernel(const CacheParams p) {
  constexpr int LPR = D / 8;
  const int part = threadIdx.x % LPR;
  const int64_t step = int64_t(gridDim.x) * (kCacheThreads / LPR);
  const int64_t first = int64_t(blockIdx.x) * (kCacheThreads / LPR) + threadIdx.x / LPR;
  for (int64_t r0 = first; r0 < p.rows; r0 += step * kCacheRows) {
    uint4 k[kCacheRows], v[kCacheRows];
    float ks[kCacheRows], vs[kCacheRows];
    bool held[kCacheRows];
#pragma unroll
    for (int i = 0; i < kCacheRows; ++i) {
      const int64_t r = r0 + i * step;
      int64_t from = -1;
      if (r < p.rows) {
        const uint32_t bh = uint32_t(r) / uint32_t(p.N), t = uint32_t(r) % uint32_t(p.N);
        const int b = bh / p.Hkv, h = bh % p.Hkv;
        if (int(t) < kv_len_of(p.pages, b)) from = cache_row(p, b, h, int(t));
      }
      held[i] = from >= 0;
      if (!held[i]) continue;
      if constexpr (E4M3) {
        const uint2 a = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.pages.K) + from * D + part * 8));
        const uint2 c = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.pages.V) + from * D + part * 8));
        k[i] = make_uint4(a.x, a.y, 0, 0);
        v[i] = make_uint4(c.x, c.y, 0, 0);
        ks[i] = __ldg(p.pages.ks + from);
        vs[i] = __ldg(p.pages.vs + from);
      } else {
        k[i] = ldg_stream_v4(static_cast<const bf16*>(p.pages.K) + from * D + part * 8);
        v[i] = ldg_stream_v4(static_cast<const bf16*>(p.pages.V) + from * D + part * 8);
      }
    }
#pragma unroll
    for (int i = 0; i < kCacheRows; ++i) {
      if (!held[i]) continue;
      const int64_t r = r0 + i * step;
      if constexpr (E4M3) {
        k[i] = restore8(make_uint2(k[i].x, k[i].y), ks[i]);
        v[i] = restore8(make_uint2(v[i].x, v[i].y), vs[i]);
      }
      *reinterpret_cast<uint4*>(p.oK + r * D + part * 8) = k[i];
      *reinterpret_cast<uint4*>(p.oV + r * D + part * 8) = v[i];
    }
  }
}

}  // namespace pisa
