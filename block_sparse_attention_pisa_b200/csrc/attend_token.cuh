// Attention of a few new tokens over a paged cache: up to 16 rows (query heads of the group
// times tokens) per key head.
//
// Bound by memory: every visible key and value is read once for all rows of its key head. The
// products run on mma.sync (m16n8k16, the 16 rows as M): with 16 rows a 128-row tcgen05 tile
// would be 7/8 empty and its hand-offs would cost more than the bytes take.
//
// No shared memory on the way in: the contraction over d may take the dimensions in any order
// (the same for Q and K), and the columns of O may stand in any order, so each lane loads 16
// contiguous bytes of a row straight into the registers that the product wants:
//   K (B operand, n = key lane/4, k = 2 (lane%4) ..): the four lanes of a key read 64 contiguous
//     bytes; Q's fragments are loaded in the same order of dimensions;
//   V (B operand, k = keys 2 (lane%4) + {0, 1, 8, 9}, n = lane/4): the eight lanes of a key read
//     128 contiguous bytes; byte permutes pair the two keys of a register.
// K of the next step is loaded once the scores of this one are in, V once its product is.
//
// In 8 bits the products run in fp16, which holds every code exactly and which a conversion
// instruction makes of two codes at once (putting codes into bf16 took more than half of the
// instructions and bound the kernel: 176 us for 519 MB; products of 8-bit operands are slower
// still, 255 us, 50 cycles each on this part's mma.sync). A power of two per row brings Q's
// largest value to [2^14, 2^15), so that values down to 2^-28 of it keep bf16's 8 bits. The
// weights (softmax weight times the value's scale) have a factor of their own per row that keeps
// the largest at 2^6 or more and below 2^15, apart from the maximum that the row's sum is
// relative to: scales of any size keep 11 bits of every weight down to 2^-20 of the largest.
// O is in that frame.
//
// The visible keys of all sequences and key heads form one list of chunks, cut evenly over
// the CTAs: sequences of different lengths balance, one long sequence fills the GPU. A CTA
// that holds a key head's whole list writes O itself; pieces go to the workspace (two slots per
// CTA) and attend_token_join_kernel adds them in order.
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "attend_tc.cuh"

namespace pisa {

struct AttendTokenParams {
  const bf16* Q;
  bf16* O;
  float* lse;
  float* part;      // fp32 [2 * ctas][16][D], then base-2 lse [2 * ctas][16]
  float* part_lse;
  Pages pages;
  int B, Hq, Hkv, N;
  int ctas;
  Window win;
  float scale;
};

constexpr int kTokenRows = 16;
constexpr int kTokenWarps = 4;

template <int D, bool E4M3>
struct AttendTokenCfg {
  static constexpr int KEYS = 2048 / D;  // of a warp's step: 16 at D = 128
  static constexpr int CHUNK = kTokenWarps * KEYS;
};

// The chunks that the new tokens of one sequence see.
struct TokenSight {
  Sight see;
  int n, nq, ns, first, chunks;
  __device__ __forceinline__ void set(const Pages& g, const Window& w, int b, int N, int chunk) {
    n = kv_len_of(g, b);
    nq = q_len_of(g, b, N);
    if (nq > 0) see.set(w, n - nq, n - 1, n);
    else see.none();
    first = see.lo / chunk;
    const int last = see.hi > see.lo ? (see.hi + chunk - 1) / chunk : first;
    ns = min((see.sk + chunk - 1) / chunk, first);
    chunks = ns + last - first;
  }
  __device__ __forceinline__ int key(int i, int chunk) const { return (i < ns ? i : first + i - ns) * chunk; }
};

// Sum of all sequences' chunks (times the key heads), and of those before sequence `want`;
// every thread gets both. Or, with want < 0, the sequence that holds unit `at` and the units
// before it.
struct UnitAt {
  long long total, before;
  int b, ctas;  // CTAs that have work: no more than there are units, so that each has some
};
template <int CHUNK>
__device__ __forceinline__ UnitAt find_unit(const AttendTokenParams& p, int want, int cta, long long* sh) {
  // each thread takes a run of sequences
  const int per = (p.B + blockDim.x - 1) / blockDim.x, b0 = min(p.B, int(threadIdx.x) * per), b1 = min(p.B, b0 + per);
  long long mine = 0;
  TokenSight s;
  for (int b = b0; b < b1; ++b) {
    s.set(p.pages, p.win, b, p.N, CHUNK);
    mine += (long long)s.chunks * p.Hkv;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, off);
    if (lane >= off) x += y;
  }
  if (lane == 31) sh[warp] = x;
  if (threadIdx.x == 0) {
    sh[kTokenWarps] = 0;
    sh[kTokenWarps + 1] = 0;
  }
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kTokenWarps; ++w) {
    if (w < warp) x += sh[w];
    total += sh[w];
  }
  const int ctas = int(total < p.ctas ? max(total, 1LL) : p.ctas);
  const long long at = total * cta / ctas;  // the CTA's first unit
  long long before = x - mine;
  for (int b = b0; b < b1; ++b) {
    s.set(p.pages, p.win, b, p.N, CHUNK);
    const long long u = (long long)s.chunks * p.Hkv;
    if (want < 0 ? (at >= before && at < before + u) : b == want) {
      sh[kTokenWarps] = before;
      sh[kTokenWarps + 1] = b;
    }
    before += u;
  }
  __syncthreads();
  return UnitAt{total, sh[kTokenWarps], int(sh[kTokenWarps + 1]), ctas};
}

__device__ __forceinline__ uint4 ldg16(const void* p, bool in) {
  uint4 r = make_uint4(0, 0, 0, 0);
  if (in) r = ldg_stream_v4(p);
  return r;
}

// Joins the four warps' sums of chunks [c0, c1) of (b, hk), in warp order: rows of O if the CTA
// holds the whole list, a piece in the workspace if not.
template <int D>
__device__ __forceinline__ void join_warps(const AttendTokenParams& p, const TokenSight& s, int b, int hk, int c0, int c1,
                                           const float (&acc)[kTokenWarps][kTokenRows][D + 4],
                                           const float (&stat)[2][kTokenWarps][kTokenRows]) {
  const int G = p.Hq / p.Hkv, rows = s.nq * G;
  const bool all = c0 == 0 && c1 == s.chunks;
  const int64_t slot = 2 * int64_t(blockIdx.x) + (c0 == 0 ? 1 : 0);
  for (int e = threadIdx.x; e < rows * (D / 4); e += 32 * kTokenWarps) {
    const int r = e / (D / 4), d = e % (D / 4) * 4;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kTokenWarps; ++w) mm = fmaxf(mm, stat[0][w][r]);
    const float m0 = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kTokenWarps; ++w) {
      const float k = tc::ex2(stat[0][w][r] - m0);  // a warp that saw nothing: 0, and its sums are 0
      const float4 y = *reinterpret_cast<const float4*>(&acc[w][r][d]);
      ll = fmaf(k, stat[1][w][r], ll);
      x.x = fmaf(k, y.x, x.x);
      x.y = fmaf(k, y.y, x.y);
      x.z = fmaf(k, y.z, x.z);
      x.w = fmaf(k, y.w, x.w);
    }
    const float inv = ll != 0.f ? 1.f / ll : 0.f;
    const float lg = ll != 0.f ? m0 + __log2f(ll) : -INFINITY;
    x = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
    if (all) {
      const size_t row = (size_t(b) * p.Hq + hk * G + r % G) * p.N + r / G;
      *reinterpret_cast<uint2*>(p.O + row * D + d) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
      if (d == 0 && p.lse) p.lse[row] = lg * 0.6931471805599453f;
    } else {
      *reinterpret_cast<float4*>(p.part + (slot * kTokenRows + r) * D + d) = x;
      if (d == 0) p.part_lse[slot * kTokenRows + r] = lg;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(32 * kTokenWarps, 2) attend_token_kernel(const AttendTokenParams p) {
  using C = AttendTokenCfg<D, false>;
  constexpr int KEYS = C::KEYS, NG = KEYS / 16, CHUNK = C::CHUNK;
  constexpr int KCH = D / 32;  // 16-byte loads of a key per lane
  constexpr int VCH = D / 64;  // ... of a value
  constexpr int KS = D / 16;                   // product steps over d
  __shared__ float acc[kTokenWarps][kTokenRows][D + 4];
  __shared__ float stat[2][kTokenWarps][kTokenRows];
  __shared__ long long sh[kTokenWarps + 2];
  asm volatile("griddepcontrol.launch_dependents;");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q = lane & 3, g = lane >> 2;
  const int G = p.Hq / p.Hkv;
  const UnitAt at = find_unit<CHUNK>(p, -1, blockIdx.x, sh);
  if (int(blockIdx.x) >= at.ctas) return;
  long long u = at.total * blockIdx.x / at.ctas;
  const long long end = at.total * (blockIdx.x + 1) / at.ctas;
  int b = at.b;
  long long before = at.before;  // units before sequence b
  TokenSight s;
  s.set(p.pages, p.win, b, p.N, CHUNK);
  const float sl2 = p.scale * 1.4426950408889634f;
  const int page_mask = (1 << p.pages.log_page) - 1;

  while (u < end) {
    while (u >= before + (long long)s.chunks * p.Hkv) {  // sequences that see nothing have no chunks
      before += (long long)s.chunks * p.Hkv;
      s.set(p.pages, p.win, ++b, p.N, CHUNK);
    }
    const int hk = int((u - before) / s.chunks), c0 = int((u - before) % s.chunks);
    const int c1 = int(min((long long)s.chunks, c0 + (end - u)));
    const int rows = s.nq * G;
    // queries, in the order of dimensions that K's loads give; and what rows g, g + 8 see
    uint32_t qa[KS][4];
    int z[2], a[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = g + 8 * h;
      const bool real = r < rows;
      const int t = real ? r / G : 0, head = hk * G + (real ? r % G : 0);
      const bf16* src = p.Q + ((size_t(b) * p.Hq + head) * p.N + t) * D;
      z[h] = max(-1, min(s.n - 1, s.n - s.nq + t + p.win.right));
      a[h] = max(0, s.n - s.nq + t - p.win.left);
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        const uint4 w = real ? __ldg(reinterpret_cast<const uint4*>(src + x * 32 + q * 8)) : make_uint4(0, 0, 0, 0);
        qa[2 * x][h] = w.x;
        qa[2 * x][2 + h] = w.y;
        qa[2 * x + 1][h] = w.z;
        qa[2 * x + 1][2 + h] = w.w;
      }
    }
    float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    uint4 kr[NG][2][KCH], vr[NG][4][VCH];
    // lane i: the page of the step's i-th group of 16 keys, -1 if none of them is seen or held
    auto pages_of = [&](int c) -> int {
      if (lane >= NG || c >= c1) return -1;
      const int j = s.key(c, CHUNK) + warp * KEYS + lane * 16;
      return s.see.any(j, 16) ? page_of(p.pages, b, j) : -1;
    };
    auto in = [&](int j) { return j < s.see.sk || (j >= s.see.lo && j < s.see.hi); };
    // `all`: every key of the step is seen by some row and held; otherwise rows that are not become 0
    auto load_k = [&](int c, int held, auto all) {
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        const int page = __shfl_sync(0xffffffffu, held, i), j = s.key(c, CHUNK) + warp * KEYS + i * 16;
        const int64_t row = ((int64_t(page) * p.Hkv + hk) << p.pages.log_page) + (j & page_mask);
        const bf16* src = static_cast<const bf16*>(p.pages.K) + (row + g) * D + q * 8;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const bool ok = all || (page >= 0 && in(j + 8 * t + g));
#pragma unroll
          for (int x = 0; x < KCH; ++x) {
            if constexpr (all) kr[i][t][x] = ldg_stream_v4(src + 8 * t * D + x * 32);
            else kr[i][t][x] = ldg16(src + 8 * t * D + x * 32, ok);
          }
        }
      }
    };
    auto load_v = [&](int c, int held, auto all) {
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        const int page = __shfl_sync(0xffffffffu, held, i), j = s.key(c, CHUNK) + warp * KEYS + i * 16;
        const int64_t row = ((int64_t(page) * p.Hkv + hk) << p.pages.log_page) + (j & page_mask);
        const bf16* src = static_cast<const bf16*>(p.pages.V) + (row + 2 * q) * D + g * 8;
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // keys 2q, 2q + 1, 2q + 8, 2q + 9
          const int key = (e & 1) + (e >> 1) * 8;
          const bool ok = all || (page >= 0 && in(j + 2 * q + key));
#pragma unroll
          for (int x = 0; x < VCH; ++x) {
            if constexpr (all) vr[i][e][x] = ldg_stream_v4(src + key * D + x * 64);
            else vr[i][e][x] = ldg16(src + key * D + x * 64, ok);
          }
        }
      }
    };
    auto full = [&](int c, int held) {
      const int j = s.key(c, CHUNK) + warp * KEYS;
      return (j + KEYS <= s.see.sk || (j >= s.see.lo && j + KEYS <= s.see.hi)) && __all_sync(0xffffffffu, lane >= NG || held >= 0);
    };
    const auto fetch_k = [&](int c, int held, bool all) {
      if (all) load_k(c, held, std::true_type{});
      else load_k(c, held, std::false_type{});
    };
    const auto fetch_v = [&](int c, int held, bool all) {
      if (all) load_v(c, held, std::true_type{});
      else load_v(c, held, std::false_type{});
    };
    int held = pages_of(c0);
    bool all = full(c0, held);
    fetch_k(c0, held, all);
    fetch_v(c0, held, all);
    int next = pages_of(c0 + 1);
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
      const int j0 = s.key(c, CHUNK) + warp * KEYS;
      float sc[NG][2][4];
#pragma unroll
      for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[i][t][e] = 0.f;
#pragma unroll
          for (int x = 0; x < KCH; ++x) {
            const uint32_t w[4] = {kr[i][t][x].x, kr[i][t][x].y, kr[i][t][x].z, kr[i][t][x].w};
            mma_bf16_16816(sc[i][t], qa[2 * x], w[0], w[1]);
            mma_bf16_16816(sc[i][t], qa[2 * x + 1], w[2], w[3]);
          }
        }
      const bool next_all = full(c + 1, next);
      if (c + 1 < c1) fetch_k(c + 1, next, next_all);
      const bool whole = all && j0 + KEYS - 1 <= s.see.p0 + p.win.right &&
                         (j0 >= s.see.p1 - p.win.left || j0 + KEYS <= p.win.sinks);
      if (!whole) {
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          const bool here = __shfl_sync(0xffffffffu, held, i) >= 0;
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = j0 + i * 16 + t * 8 + 2 * q + (e & 1), h = e >> 1;
              if (!(here && j <= z[h] && (j >= a[h] || j < p.win.sinks))) sc[i][t][e] = -INFINITY;
            }
        }
      }
      bool move = false;
      float f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
          for (int t = 0; t < 2; ++t) mx = fmaxf(mx, fmaxf(sc[i][t][2 * h], sc[i][t][2 * h + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * sl2;
        f[h] = 1.f;
        if (mx > m[h] + 8.f) {  // the accumulator follows the maximum in steps of 2^8 or more
          if (m[h] != -INFINITY) {
            f[h] = tc::ex2(m[h] - mx);
            move = true;
          }
          m[h] = mx;
        }
      }
      if (__any_sync(0xffffffffu, move)) {
        l[0] *= f[0];
        l[1] *= f[1];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][0] *= f[0];
          o[i][1] *= f[0];
          o[i][2] *= f[1];
          o[i][3] *= f[1];
        }
      }
      const float n0 = m[0] == -INFINITY ? 0.f : -m[0], n1 = m[1] == -INFINITY ? 0.f : -m[1];
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        uint32_t pa[4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = tc::ex2(fmaf(sc[i][t][e], sl2, e < 2 ? n0 : n1));
          l[0] += w[0] + w[1];
          l[1] += w[2] + w[3];
          pa[2 * t] = pack_bf16x2(w[0], w[1]);
          pa[2 * t + 1] = pack_bf16x2(w[2], w[3]);
        }
        // column e of a lane's chunk x is one product's column g: d = 64 x + 8 g + e
#pragma unroll
        for (int x = 0; x < VCH; ++x) {
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = y == 0 ? vr[i][e][x].x : y == 1 ? vr[i][e][x].y : y == 2 ? vr[i][e][x].z : vr[i][e][x].w;
            mma_bf16_16816(o[8 * x + 2 * y], pa, __byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410));
            mma_bf16_16816(o[8 * x + 2 * y + 1], pa, __byte_perm(w[0], w[1], 0x7632), __byte_perm(w[2], w[3], 0x7632));
          }
        }
      }
      if (c + 1 < c1) fetch_v(c + 1, next, next_all);
      held = next;
      all = next_all;
      next = pages_of(c + 2);
    }
    // the warps' accumulators, joined in warp order
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
    __syncthreads();  // the previous key head's joined rows have been read
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int col = 2 * q + (e & 1);  // column of product i
        const int d = (i >> 3) * 64 + col * 8 + (i & 7);
        acc[warp][g + 8 * (e >> 1)][d] = o[i][e];
      }
    if (q == 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        stat[0][warp][g + 8 * h] = m[h];
        stat[1][warp][g + 8 * h] = l[h];
      }
    }
    __syncthreads();
    join_warps<D>(p, s, b, hk, c0, c1, acc, stat);
    u += c1 - c0;
  }
}

// the power of two with these bits in its fp32 exponent field
__device__ __forceinline__ float exponent(int field) { return __uint_as_float(uint32_t(field) << 23); }

// D = A(16x16 fp16, row) * B(16x8 fp16, col) + D, fp32 accumulate.
__device__ __forceinline__ void mma_f16_16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The low (high) two e4m3 codes of a word -> two fp16, exact (codes of NaN too).
__device__ __forceinline__ uint32_t codes_to_f16_lo(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t codes_to_f16_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  __half2 r = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&r);
}

template <int D>
__global__ void __launch_bounds__(32 * kTokenWarps, 3) attend_token8_kernel(const AttendTokenParams p) {
  using C = AttendTokenCfg<D, true>;
  constexpr int KEYS = C::KEYS, NG = KEYS / 16, CHUNK = C::CHUNK;
  constexpr int KCH = D / 64;  // 16-byte loads of a key per lane, four product steps each
  constexpr int W = D / 32;    // words of a value per lane
  __shared__ float acc[kTokenWarps][kTokenRows][D + 4];
  __shared__ float stat[2][kTokenWarps][kTokenRows];
  __shared__ long long sh[kTokenWarps + 2];
  asm volatile("griddepcontrol.launch_dependents;");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int q = lane & 3, gr = lane >> 2;
  const int G = p.Hq / p.Hkv;
  const UnitAt at = find_unit<CHUNK>(p, -1, blockIdx.x, sh);
  if (int(blockIdx.x) >= at.ctas) return;
  long long u = at.total * blockIdx.x / at.ctas;
  const long long end = at.total * (blockIdx.x + 1) / at.ctas;
  int b = at.b;
  long long before = at.before;  // units before sequence b
  TokenSight s;
  s.set(p.pages, p.win, b, p.N, CHUNK);
  const int page_mask = (1 << p.pages.log_page) - 1;

  while (u < end) {
    while (u >= before + (long long)s.chunks * p.Hkv) {  // sequences that see nothing have no chunks
      before += (long long)s.chunks * p.Hkv;
      s.set(p.pages, p.win, ++b, p.N, CHUNK);
    }
    const int hk = int((u - before) / s.chunks), c0 = int((u - before) % s.chunks);
    const int c1 = int(min((long long)s.chunks, c0 + (end - u)));
    const int rows = s.nq * G;
    // queries, in the order of dimensions that K's loads give: step 4 x + y has the lane's
    // dimensions 64 x + 16 q + 4 y + {0 .. 3}
    uint32_t qa[D / 16][4];
    int z[2], a[2];
    float sl2[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = gr + 8 * h;
      const bool real = r < rows;
      const int t = real ? r / G : 0, head = hk * G + (real ? r % G : 0);
      const bf16* src = p.Q + ((size_t(b) * p.Hq + head) * p.N + t) * D;
      z[h] = max(-1, min(s.n - 1, s.n - s.nq + t + p.win.right));
      a[h] = max(0, s.n - s.nq + t - p.win.left);
      uint4 w[D / 32];
      uint32_t top = 0;
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        w[x] = real ? __ldg(reinterpret_cast<const uint4*>(src + (x >> 1) * 64 + q * 16 + (x & 1) * 8)) : make_uint4(0, 0, 0, 0);
        const uint32_t ww[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) top = max(top, max(ww[i] & 0x7fffu, (ww[i] >> 16) & 0x7fffu));
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int field = min(253, 268 - int(top >> 7));  // top * 2^(field - 127) lies in [2^14, 2^15)
      const float up = top >= 0x7f80u ? __uint_as_float(0x7fc00000u) : exponent(field);  // a NaN or infinity: NaN
      sl2[h] = p.scale * 1.4426950408889634f * exponent(254 - field);
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        qa[2 * x][h] = pack_f16x2(bf16_lo(w[x].x) * up, bf16_hi(w[x].x) * up);
        qa[2 * x][2 + h] = pack_f16x2(bf16_lo(w[x].y) * up, bf16_hi(w[x].y) * up);
        qa[2 * x + 1][h] = pack_f16x2(bf16_lo(w[x].z) * up, bf16_hi(w[x].z) * up);
        qa[2 * x + 1][2 + h] = pack_f16x2(bf16_lo(w[x].w) * up, bf16_hi(w[x].w) * up);
      }
    }
    float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    constexpr int kTopField = 247;  // g is at most 2^120
    float f[2] = {exponent(kTopField), exponent(kTopField)};  // g of either row
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    // product column gr of n-tile t is key 8 t + gr of its group of 16; the lane's weights belong to
    // keys 8 t + 2 q + {0, 1}, so those are the rows of V that it loads
    uint4 kr[NG][2][KCH];
    uint32_t vr[NG][2][2][W];
    float2 ks[NG][2], vs[NG][2];
    // lane i: the page of the step's i-th group of 16 keys, -1 if none of them is seen or held
    auto pages_of = [&](int c) -> int {
      if (lane >= NG || c >= c1) return -1;
      const int j = s.key(c, CHUNK) + warp * KEYS + lane * 16;
      return s.see.any(j, 16) ? page_of(p.pages, b, j) : -1;
    };
    auto in = [&](int j) { return j < s.see.sk || (j >= s.see.lo && j < s.see.hi); };
    auto row_of = [&](int page, int j) {
      return ((int64_t(page) * p.Hkv + hk) << p.pages.log_page) + (j & page_mask);
    };
    // `all`: every key of the step is seen by some row and held; otherwise rows that are not become 0
    auto load_k = [&](int c, int held, auto all) {
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        const int page = __shfl_sync(0xffffffffu, held, i), j = s.key(c, CHUNK) + warp * KEYS + i * 16;
        const int64_t row = row_of(page, j);
        const uint8_t* src = static_cast<const uint8_t*>(p.pages.K) + (row + gr) * D + q * 16;
        const float* sp = p.pages.ks + row + 2 * q;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const bool ok = all || (page >= 0 && in(j + 8 * t + gr));
#pragma unroll
          for (int x = 0; x < KCH; ++x) {
            if constexpr (all) kr[i][t][x] = ldg_stream_v4(src + 8 * t * D + x * 64);
            else kr[i][t][x] = ldg16(src + 8 * t * D + x * 64, ok);
          }
          ks[i][t] = all || page >= 0 ? __ldg(reinterpret_cast<const float2*>(sp + 8 * t)) : make_float2(0.f, 0.f);
        }
      }
    };
    auto load_v = [&](int c, int held, auto all) {
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        const int page = __shfl_sync(0xffffffffu, held, i), j = s.key(c, CHUNK) + warp * KEYS + i * 16 + 2 * q;
        const int64_t row = row_of(page, j);
        const uint8_t* src = static_cast<const uint8_t*>(p.pages.V) + row * D + gr * (D / 8);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const bool ok[2] = {all || (page >= 0 && in(j + 8 * t)), all || (page >= 0 && in(j + 8 * t + 1))};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if constexpr (D == 128) {
              uint4 w;
              if constexpr (all) w = ldg_stream_v4(src + (8 * t + e) * D);
              else w = ldg16(src + (8 * t + e) * D, ok[e]);
              vr[i][t][e][0] = w.x;
              vr[i][t][e][1] = w.y;
              vr[i][t][e][W - 2] = w.z;
              vr[i][t][e][W - 1] = w.w;
            } else {
              const uint2 w = ok[e] ? __ldg(reinterpret_cast<const uint2*>(src + (8 * t + e) * D)) : make_uint2(0, 0);
              vr[i][t][e][0] = w.x;
              vr[i][t][e][1] = w.y;
            }
          }
          const float2 x = all || page >= 0 ? __ldg(reinterpret_cast<const float2*>(p.pages.vs + row + 8 * t)) : make_float2(0.f, 0.f);
          vs[i][t] = make_float2(ok[0] ? x.x : 0.f, ok[1] ? x.y : 0.f);
        }
      }
    };
    auto full = [&](int c, int held) {
      const int j = s.key(c, CHUNK) + warp * KEYS;
      return (j + KEYS <= s.see.sk || (j >= s.see.lo && j + KEYS <= s.see.hi)) && __all_sync(0xffffffffu, lane >= NG || held >= 0);
    };
    const auto fetch_k = [&](int c, int held, bool all) {
      if (all) load_k(c, held, std::true_type{});
      else load_k(c, held, std::false_type{});
    };
    const auto fetch_v = [&](int c, int held, bool all) {
      if (all) load_v(c, held, std::true_type{});
      else load_v(c, held, std::false_type{});
    };
    int held = pages_of(c0);
    bool all = full(c0, held);
    fetch_k(c0, held, all);
    fetch_v(c0, held, all);
    int next = pages_of(c0 + 1);
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
      const int j0 = s.key(c, CHUNK) + warp * KEYS;
      float sc[NG][2][4];
#pragma unroll
      for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[i][t][e] = 0.f;
#pragma unroll
          for (int x = 0; x < KCH; ++x) {
            const uint32_t w[4] = {kr[i][t][x].x, kr[i][t][x].y, kr[i][t][x].z, kr[i][t][x].w};
#pragma unroll
            for (int y = 0; y < 4; ++y)
              mma_f16_16816(sc[i][t], qa[4 * x + y], codes_to_f16_lo(w[y]), codes_to_f16_hi(w[y]));
          }
          sc[i][t][0] *= ks[i][t].x;
          sc[i][t][1] *= ks[i][t].y;
          sc[i][t][2] *= ks[i][t].x;
          sc[i][t][3] *= ks[i][t].y;
        }
      const bool next_all = full(c + 1, next);
      if (c + 1 < c1) fetch_k(c + 1, next, next_all);
      const bool whole = all && j0 + KEYS - 1 <= s.see.p0 + p.win.right &&
                         (j0 >= s.see.p1 - p.win.left || j0 + KEYS <= p.win.sinks);
      if (!whole) {
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          const bool here = __shfl_sync(0xffffffffu, held, i) >= 0;
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = j0 + i * 16 + t * 8 + 2 * q + (e & 1), h = e >> 1;
              if (!(here && j <= z[h] && (j >= a[h] || j < p.win.sinks))) sc[i][t][e] = -INFINITY;
            }
        }
      }
      float old[2], tm[2] = {0.f, 0.f};  // g in the new frame of m, before it is bounded; largest weight
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
          for (int t = 0; t < 2; ++t) mx = fmaxf(mx, fmaxf(sc[i][t][2 * h], sc[i][t][2 * h + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * sl2[h];
        old[h] = f[h];
        if (mx > m[h] + 8.f) {  // the sum follows the maximum in steps of 2^8 or more
          if (m[h] != -INFINITY) {
            l[h] *= tc::ex2(m[h] - mx);
            old[h] *= tc::ex2(mx - m[h]);  // infinity: what O holds no longer counts
          }
          m[h] = mx;
        }
      }
      const float neg[2] = {m[0] == -INFINITY ? 0.f : -m[0], m[1] == -INFINITY ? 0.f : -m[1]};
#pragma unroll
      for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int h = e >> 1;
            const float w = tc::ex2(fmaf(sc[i][t][e], sl2[h], neg[h]));
            l[h] += w;
            sc[i][t][e] = w * (e & 1 ? vs[i][t].y : vs[i][t].x);
            tm[h] = fmaxf(tm[h], sc[i][t][e]);
          }
      float r[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        tm[h] = fmaxf(tm[h], __shfl_xor_sync(0xffffffffu, tm[h], 1));
        tm[h] = fmaxf(tm[h], __shfl_xor_sync(0xffffffffu, tm[h], 2));
        // the largest weight passes 2^15: bring it to [2^6, 2^7)
        f[h] = tm[h] * old[h] > 32768.f ? exponent(min(kTopField, 260 - int(__float_as_uint(tm[h]) >> 23)))
                                        : fminf(old[h], exponent(kTopField));
        r[h] = f[h] == old[h] ? 1.f : __fdividef(f[h], old[h]);
        if (old[h] > 1e37f) r[h] = f[h] == old[h] ? 1.f : 0.f;
      }
      if (__any_sync(0xffffffffu, r[0] != 1.f || r[1] != 1.f)) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          o[i][0] *= r[0];
          o[i][1] *= r[0];
          o[i][2] *= r[1];
          o[i][3] *= r[1];
        }
      }
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        uint32_t pa[4];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h) pa[2 * t + h] = pack_f16x2(sc[i][t][2 * h] * f[h], sc[i][t][2 * h + 1] * f[h]);
        // byte e of word x of the lane's codes is column gr of product 4 x + e: d = gr D/8 + 4 x + e
#pragma unroll
        for (int x = 0; x < W; ++x) {
          const uint32_t lo0 = __byte_perm(vr[i][0][0][x], vr[i][0][1][x], 0x5140), hi0 = __byte_perm(vr[i][0][0][x], vr[i][0][1][x], 0x7362);
          const uint32_t lo1 = __byte_perm(vr[i][1][0][x], vr[i][1][1][x], 0x5140), hi1 = __byte_perm(vr[i][1][0][x], vr[i][1][1][x], 0x7362);
          mma_f16_16816(o[4 * x], pa, codes_to_f16_lo(lo0), codes_to_f16_lo(lo1));
          mma_f16_16816(o[4 * x + 1], pa, codes_to_f16_hi(lo0), codes_to_f16_hi(lo1));
          mma_f16_16816(o[4 * x + 2], pa, codes_to_f16_lo(hi0), codes_to_f16_lo(hi1));
          mma_f16_16816(o[4 * x + 3], pa, codes_to_f16_hi(hi0), codes_to_f16_hi(hi1));
        }
      }
      if (c + 1 < c1) fetch_v(c + 1, next, next_all);
      held = next;
      all = next_all;
      next = pages_of(c + 2);
    }
    // the warps' accumulators, joined in warp order
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      f[h] = 1.f / f[h];
    }
    __syncthreads();  // the previous key head's joined rows have been read
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        acc[warp][gr + 8 * (e >> 1)][(2 * q + (e & 1)) * (D / 8) + i] = o[i][e] * f[e >> 1];
    if (q == 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        stat[0][warp][gr + 8 * h] = m[h];
        stat[1][warp][gr + 8 * h] = l[h];
      }
    }
    __syncthreads();
    join_warps<D>(p, s, b, hk, c0, c1, acc, stat);
    u += c1 - c0;
  }
}

// One block per sequence and key head: joins the pieces that several CTAs hold, in order, and
// writes the rows of sequences that see nothing.
template <int D, bool E4M3>
__global__ void __launch_bounds__(32 * kTokenWarps) attend_token_join_kernel(const AttendTokenParams p) {
  constexpr int CHUNK = AttendTokenCfg<D, E4M3>::CHUNK;
  __shared__ long long sh[kTokenWarps + 2];
  const int b = blockIdx.x / p.Hkv, hk = blockIdx.x % p.Hkv, G = p.Hq / p.Hkv;
  const UnitAt at = find_unit<CHUNK>(p, b, 0, sh);
  TokenSight s;
  s.set(p.pages, p.win, b, p.N, CHUNK);
  const long long u0 = at.before + (long long)hk * s.chunks, u1 = u0 + s.chunks;
  // the CTA that holds unit u is the last one whose first unit is not behind it
  const long long first = s.chunks ? ((u0 + 1) * at.ctas - 1) / at.total : 0;
  const long long last = s.chunks ? (u1 * at.ctas - 1) / at.total : -1;
  // every block waits, so that this grid does not end before the one it depends on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (first == last) return;
  for (int e = threadIdx.x; e < s.nq * G * (D / 4); e += 32 * kTokenWarps) {
    const int r = e / (D / 4), d = e % (D / 4) * 4;
    float m = -INFINITY;
    for (long long c = first; c <= last; ++c) m = fmaxf(m, p.part_lse[(2 * c + (c == first)) * kTokenRows + r]);
    const float m0 = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (long long c = first; c <= last; ++c) {
      const int64_t row = (2 * c + (c == first)) * kTokenRows + r;
      const float w = tc::ex2(p.part_lse[row] - m0);
      const float4 y = *reinterpret_cast<const float4*>(p.part + row * D + d);
      l += w;
      x.x = fmaf(w, y.x, x.x);
      x.y = fmaf(w, y.y, x.y);
      x.z = fmaf(w, y.z, x.z);
      x.w = fmaf(w, y.w, x.w);
    }
    const float inv = l != 0.f ? 1.f / l : 0.f;
    const size_t row = (size_t(b) * p.Hq + hk * G + r % G) * p.N + r / G;
    *reinterpret_cast<uint2*>(p.O + row * D + d) = make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
    if (d == 0 && p.lse) p.lse[row] = l != 0.f ? (m0 + __log2f(l)) * 0.6931471805599453f : -INFINITY;
  }
}

}  // namespace pisa
