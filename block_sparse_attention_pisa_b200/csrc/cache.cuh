// Paged key/value cache: rows are quantised as they are written, and read back.
//
// A row is one token of one key head (d values). In 8 bits it is held as e4m3 codes with one
// fp32 scale: scale = max(amax|x| / 448, 2^-126), code = e4m3(x / scale) (the fp32 quotient,
// rounded to nearest even), and read back as bf16(code * scale). The bits of |x| grow with
// |x| and a NaN's lie above infinity's, so the maximum is taken over the bits: a row with an
// infinity or a NaN gets the scale NaN, and the whole row reads back as NaN.
//
// Both kernels are bound by memory: each row of x is read once and its codes written once (or
// the reverse). A thread takes 16 bytes of the cache's row (16 codes or 8 bf16) of K and of V,
// kCacheRows rows in flight.
#pragma once

#include "window.cuh"

namespace pisa {

constexpr int kCacheThreads = 256;
constexpr int kCacheRows = 2;  // rows of K and of V in flight per thread

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

template <int D, bool E4M3>
struct CacheCfg {
  static constexpr int PER = E4M3 ? 16 : 8;        // values of a row per thread
  static constexpr int LPR = D / PER;              // threads per row
  static constexpr int ROWS = kCacheThreads / LPR; // rows of a CTA's step
};

// cache row of position `pos` of (b, h), or -1
__device__ __forceinline__ int64_t cache_row(const CacheParams& p, int b, int h, int pos) {
  const int at = page_of(p.pages, b, pos);
  return at < 0 ? -1 : ((int64_t(at) * p.Hkv + h) << p.pages.log_page) + (pos & ((1 << p.pages.log_page) - 1));
}

// four quotients -> four codes
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  return uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3)) |
         uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3)) << 16;
}

// 16 bf16 of a row -> its scale and 16 codes.
// The fp32 quotient x / scale by Markstein's correction (P. Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990): with y the correctly
// rounded reciprocal and q = x y, the remainder r = x - q scale is exact and q + r y is the
// correctly rounded quotient, unless scale's mantissa is all ones or r leaves the range. Rows
// of such scales (below 2^-90 the remainder could) divide. Three operations a value; with a
// division for each the kernel was bound by issue (75 us for 2 x 24 x 4096 rows of 128).
template <int LPR>
__device__ __forceinline__ uint4 quantise16(const uint4& x0, const uint4& x1, float& scale) {
  const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
#pragma unroll
  for (int off = 1; off < LPR; off <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
  if (top >= 0x7f80u) top = 0x7fc0u;  // an infinity or a NaN: NaN for the row
  scale = __fdiv_rn(__uint_as_float(top << 16), 448.f);
  if (scale < 1.17549435e-38f) scale = 1.17549435e-38f;  // a NaN stays one
  const bool divide = scale < 8.0779357e-28f || (__float_as_uint(scale) & 0x7fffffu) == 0x7fffffu;
  uint32_t c[4];
  if (!divide) {
    const float y = __frcp_rn(scale);
    auto quotient = [&](float x) {
      const float q = x * y;
      return fmaf(fmaf(-q, scale, x), y, q);
    };
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = codes4(quotient(bf16_lo(w[2 * i])), quotient(bf16_hi(w[2 * i])), quotient(bf16_lo(w[2 * i + 1])),
                    quotient(bf16_hi(w[2 * i + 1])));
  } else {
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {  // rolled: rare, and its code should stay small
      const uint32_t a = i == 0 ? w[0] : i == 1 ? w[2] : i == 2 ? w[4] : w[6];
      const uint32_t b = i == 0 ? w[1] : i == 1 ? w[3] : i == 2 ? w[5] : w[7];
      const uint32_t x = codes4(__fdiv_rn(bf16_lo(a), scale), __fdiv_rn(bf16_hi(a), scale), __fdiv_rn(bf16_lo(b), scale),
                                __fdiv_rn(bf16_hi(b), scale));
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k == i) c[k] = x;
    }
  }
  return make_uint4(c[0], c[1], c[2], c[3]);
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kCacheThreads) cache_write_kernel(const CacheParams p) {
  using C = CacheCfg<D, E4M3>;
  constexpr int X = C::PER / 8;  // 16-byte loads of a row per thread
  const int part = threadIdx.x % C::LPR, mine = threadIdx.x / C::LPR;
  const int64_t step = int64_t(gridDim.x) * C::ROWS;
  // every thread of a warp takes the same number of rounds (the shuffles need all lanes)
  for (int64_t r0 = int64_t(blockIdx.x) * C::ROWS; r0 < p.rows; r0 += step * kCacheRows) {
    uint4 k[kCacheRows][X], v[kCacheRows][X];
    int64_t to[kCacheRows];
    // the values do not wait for the lengths and the table: a token that turns out not to be
    // real is read all the same (it lies inside K and V)
#pragma unroll
    for (int i = 0; i < kCacheRows; ++i) {
      const int64_t r = r0 + mine + i * step;
#pragma unroll
      for (int x = 0; x < X; ++x) {
        k[i][x] = v[i][x] = make_uint4(0, 0, 0, 0);
        if (r < p.rows) {
          k[i][x] = ldg_stream_v4(p.K + r * D + part * C::PER + x * 8);
          v[i][x] = ldg_stream_v4(p.V + r * D + part * C::PER + x * 8);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kCacheRows; ++i) {
      const int64_t r = r0 + mine + i * step;
      to[i] = -1;
      if (r < p.rows) {
        const uint32_t bh = uint32_t(r) / uint32_t(p.N), t = uint32_t(r) % uint32_t(p.N);
        const int b = bh / p.Hkv, h = bh % p.Hkv;
        const int n = q_len_of(p.pages, b, p.N), pos = kv_len_of(p.pages, b) - n + int(t);
        if (int(t) < n && pos >= 0) to[i] = cache_row(p, b, h, pos);
      }
    }
#pragma unroll
    for (int i = 0; i < kCacheRows; ++i) {
      if constexpr (E4M3) {
        float ks, vs;
        const uint4 kc = quantise16<C::LPR>(k[i][0], k[i][1], ks), vc = quantise16<C::LPR>(v[i][0], v[i][1], vs);
        if (to[i] >= 0) {
          *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.cK) + to[i] * D + part * 16) = kc;
          *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.cV) + to[i] * D + part * 16) = vc;
          if (part == 0) {
            p.ks[to[i]] = ks;
            p.vs[to[i]] = vs;
          }
        }
      } else if (to[i] >= 0) {
        *reinterpret_cast<uint4*>(static_cast<bf16*>(p.cK) + to[i] * D + part * 8) = k[i][0];
        *reinterpret_cast<uint4*>(static_cast<bf16*>(p.cV) + to[i] * D + part * 8) = v[i][0];
      }
    }
  }
}

// 8 codes and their scale -> 8 bf16
__device__ __forceinline__ uint4 restore8(uint32_t lo, uint32_t hi, float scale) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t two = e4m3x2_to_bf16x2((i < 2 ? lo : hi) >> (16 * (i & 1)));
    w[i] = pack_bf16x2(bf16_lo(two) * scale, bf16_hi(two) * scale);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kCacheThreads) cache_read_kernel(const CacheParams p) {
  using C = CacheCfg<D, E4M3>;
  const int part = threadIdx.x % C::LPR;
  const int64_t step = int64_t(gridDim.x) * C::ROWS;
  for (int64_t r0 = int64_t(blockIdx.x) * C::ROWS + threadIdx.x / C::LPR; r0 < p.rows; r0 += step * kCacheRows) {
    uint4 k[kCacheRows], v[kCacheRows];
    float ks[kCacheRows], vs[kCacheRows];
    int64_t from[kCacheRows];
#pragma unroll
    for (int i = 0; i < kCacheRows; ++i) {
      const int64_t r = r0 + i * step;
      from[i] = -1;
      if (r < p.rows) {
        const uint32_t bh = uint32_t(r) / uint32_t(p.N), t = uint32_t(r) % uint32_t(p.N);
        const int b = bh / p.Hkv, h = bh % p.Hkv;
        if (int(t) < kv_len_of(p.pages, b)) from[i] = cache_row(p, b, h, int(t));
      }
    }
#pragma unroll
    for (int i = 0; i < kCacheRows; ++i) {
      if (from[i] < 0) continue;
      k[i] = ldg_stream_v4(static_cast<const uint8_t*>(p.pages.K) + from[i] * (E4M3 ? D : 2 * D) + part * 16);
      v[i] = ldg_stream_v4(static_cast<const uint8_t*>(p.pages.V) + from[i] * (E4M3 ? D : 2 * D) + part * 16);
      if constexpr (E4M3) {
        ks[i] = __ldg(p.pages.ks + from[i]);
        vs[i] = __ldg(p.pages.vs + from[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < kCacheRows; ++i) {
      if (from[i] < 0) continue;
      uint4* dk = reinterpret_cast<uint4*>(p.oK + (r0 + i * step) * D + part * C::PER);
      uint4* dv = reinterpret_cast<uint4*>(p.oV + (r0 + i * step) * D + part * C::PER);
      if constexpr (E4M3) {
        dk[0] = restore8(k[i].x, k[i].y, ks[i]);
        dk[1] = restore8(k[i].z, k[i].w, ks[i]);
        dv[0] = restore8(v[i].x, v[i].y, vs[i]);
        dv[1] = restore8(v[i].z, v[i].w, vs[i]);
      } else {
        dk[0] = k[i];
        dv[0] = v[i];
      }
    }
  }
}

}  // namespace pisa
