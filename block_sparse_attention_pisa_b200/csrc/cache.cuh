// Paged key/value cache: rows are quantised as they are written, and read back.
//
// A row is one token of one key head (d values). In 8 bits it is held as e4m3 codes with one
// fp32 scale: scale = max(amax|x| / 448, 2^-126), code = e4m3(x / scale) (the fp32 quotient,
// rounded to nearest even), and read back as bf16(code * scale). The bits of |x| grow with
// |x| and a NaN's lie above infinity's, so the maximum is taken over the bits: a row with an
// infinity or a NaN gets the scale NaN, and the whole row reads back as NaN.
//
// Both kernels read each row of x once and write its codes once (or the reverse). Reading back, and
// bf16 both ways, a thread takes 16 bytes of the cache's row of K and of V, kCacheRows rows in
// flight, and memory bounds it (126 us for 8 x 8 sequences of 9-16 K rows of 128: 5.1 TB/s, two
// thirds of it writes; 131 us without streaming stores, 140 and 149 us with one and four rows in
// flight; in bf16 144 us, 5.8 TB/s; written in bf16, 2 x 24 x 4096 rows 37 us, 5.4 TB/s). Quantising, a
// thread takes 32 values.
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

// The fp32 quotient a / b by Markstein's correction (P. Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990): with y the correctly rounded
// reciprocal of b and q = a y, the remainder r = a - q b is exact and q + r y is the correctly
// rounded quotient, unless b's mantissa is all ones or r leaves the range.
__device__ __forceinline__ float quotient(float a, float b, float y) {
  const float q = a * y;
  return fmaf(fmaf(-q, b, a), y, q);
}

// 32 bf16 of a row -> its scale and 32 codes. Three operations a value; rows whose scale Markstein's
// correction does not cover (below 2^-90 its remainder could leave the range) divide. With a
// division for each value the kernel was bound by issue (75 us for 2 x 24 x 4096 rows of 128), and
// still was (50 us) with 16 values per thread, where the row's own work weighs twice as much. Now (32 us,
// 4.7 TB/s, issue slots half used) it waits: a thread has one row's loads in flight, and asks for the
// next once it has stored this one.
template <int LPR>
__device__ __forceinline__ void quantise32(const uint4 (&x)[4], float& scale, uint4 (&code)[2]) {
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[4 * i] = x[i].x;
    w[4 * i + 1] = x[i].y;
    w[4 * i + 2] = x[i].z;
    w[4 * i + 3] = x[i].w;
  }
  uint32_t top = 0;  // the maximum over the bits, a half of the word at a time
#pragma unroll
  for (int i = 0; i < 16; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
  top = max(top & 0xffffu, top >> 16);
#pragma unroll
  for (int off = 1; off < LPR; off <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, off));
  if (top >= 0x7f80u) top = 0x7fc0u;  // an infinity or a NaN: NaN for the row
  const float amax = __uint_as_float(top << 16);
  scale = quotient(amax, 448.f, 1.f / 448.f);
  bool divide = scale < 8.0779357e-28f;  // 2^-90
  if (divide) {
    scale = __fdiv_rn(amax, 448.f);
    if (scale < 1.17549435e-38f) scale = 1.17549435e-38f;
  }
  divide |= (__float_as_uint(scale) & 0x7fffffu) == 0x7fffffu;
  uint32_t c[8];
  if (!divide) {
    const float y = __frcp_rn(scale);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      c[i] = codes4(quotient(bf16_lo(w[2 * i]), scale, y), quotient(bf16_hi(w[2 * i]), scale, y),
                    quotient(bf16_lo(w[2 * i + 1]), scale, y), quotient(bf16_hi(w[2 * i + 1]), scale, y));
  } else {
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {  // rolled: rare, and its code should stay small
      uint32_t a = 0, b = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k == i) {
          a = w[2 * k];
          b = w[2 * k + 1];
        }
      const uint32_t v = codes4(__fdiv_rn(bf16_lo(a), scale), __fdiv_rn(bf16_hi(a), scale), __fdiv_rn(bf16_lo(b), scale),
                                __fdiv_rn(bf16_hi(b), scale));
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k == i) c[k] = v;
    }
  }
  code[0] = make_uint4(c[0], c[1], c[2], c[3]);
  code[1] = make_uint4(c[4], c[5], c[6], c[7]);
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kCacheThreads) cache_write_kernel(const CacheParams p) {
  constexpr int PER = E4M3 ? 32 : 8, LPR = D / PER, ROWS = kCacheThreads / LPR;  // values, threads of a row; rows of a CTA
  constexpr int FLY = E4M3 ? 1 : kCacheRows, X = PER / 8;  // rows in flight, 16-byte loads of each
  const int part = threadIdx.x % LPR, mine = threadIdx.x / LPR;
  const int64_t step = int64_t(gridDim.x) * ROWS;
  // every thread of a warp takes the same number of rounds (the shuffles need all lanes)
  for (int64_t r0 = int64_t(blockIdx.x) * ROWS; r0 < p.rows; r0 += step * FLY) {
    uint4 k[FLY][X], v[FLY][X];
    int64_t to[FLY];
    // the values do not wait for the lengths and the table: a token that turns out not to be
    // real is read all the same (it lies inside K and V)
#pragma unroll
    for (int i = 0; i < FLY; ++i) {
      const int64_t r = r0 + mine + i * step;
#pragma unroll
      for (int x = 0; x < X; ++x) {
        k[i][x] = v[i][x] = make_uint4(0, 0, 0, 0);
        if (r < p.rows) {
          k[i][x] = ldg_stream_v4(p.K + r * D + part * PER + x * 8);
          v[i][x] = ldg_stream_v4(p.V + r * D + part * PER + x * 8);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < FLY; ++i) {
      const int64_t r = r0 + mine + i * step;
      to[i] = -1;
      if (r < p.rows) {
        const uint32_t bh = uint32_t(r) / uint32_t(p.N), t = uint32_t(r) - bh * uint32_t(p.N);
        const int b = bh / p.Hkv, h = bh - b * p.Hkv;
        const int n = q_len_of(p.pages, b, p.N), pos = kv_len_of(p.pages, b) - n + int(t);
        if (int(t) < n && pos >= 0) to[i] = cache_row(p, b, h, pos);
      }
    }
#pragma unroll
    for (int i = 0; i < FLY; ++i) {
      if constexpr (E4M3) {
        float ks, vs;
        uint4 kc[2], vc[2];
        quantise32<LPR>(k[i], ks, kc);
        quantise32<LPR>(v[i], vs, vc);
        if (to[i] >= 0) {
          uint4* dk = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.cK) + to[i] * D + part * 32);
          uint4* dv = reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.cV) + to[i] * D + part * 32);
          dk[0] = kc[0];
          dk[1] = kc[1];
          dv[0] = vc[0];
          dv[1] = vc[1];
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
        __stcs(&dk[0], restore8(k[i].x, k[i].y, ks[i]));
        __stcs(&dk[1], restore8(k[i].z, k[i].w, ks[i]));
        __stcs(&dv[0], restore8(v[i].x, v[i].y, vs[i]));
        __stcs(&dv[1], restore8(v[i].z, v[i].w, vs[i]));
      } else {
        __stcs(&dk[0], k[i]);
        __stcs(&dv[0], v[i]);
      }
    }
  }
}

}  // namespace pisa
