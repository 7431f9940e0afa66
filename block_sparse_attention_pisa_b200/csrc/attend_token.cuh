// Attention of a few new tokens over a paged cache: up to 16 rows (query heads of the group
// times tokens) per key head.
//
// Bound by memory: every visible key and value is read once for all rows of its key head. The
// products run on mma.sync (m16n8k16) transposed, S^T = K Q^T and O^T = V^T P^T: keys (and then
// dimensions) fill the 16 rows of the first operand, the query rows are its 8 columns (NR = 2:
// two products). With a 128-row tcgen05 tile 7/8 of it would be empty and its hand-offs would
// cost more than the bytes take; with the query rows as M of m16n8k16, half of every fragment
// and of the softmax's work would be padding at 8 rows or fewer (4 sequences of 47-76 K tokens, 8
// key heads of 128 in 8 bits, 5 rows each: 147 us, transposed 102 us at 5.1 TB/s; 32 sequences
// of 4-8 K in bf16, 4 rows each: 145 and 129 us at 6.3 TB/s, the copy rate).
//
// No shared memory on the way in: the contraction over d may take the dimensions in any order
// (the same for Q and K), and the rows of O^T may stand in any order, so each lane loads 16
// contiguous bytes of a row straight into the registers that the product wants:
//   K (rows = keys lane/4 and 8 + lane/4): the four lanes of a key read 64 contiguous bytes;
//     Q's fragments are loaded in the same order of dimensions;
//   V (contraction over keys 2 (lane%4) + {0, 1, 8, 9}): the eight lanes of a key read 128
//     contiguous bytes; byte permutes pair the two keys of a register.
// P^T comes out of S^T with one 8 x 8 transposition (movmatrix) per 8 keys. K of the next step is
// loaded once the scores of this one are in, V once its product is. The running maximum of a row
// is looked at by a vote: lanes exchange maxima only when one of them passes the current one by
// more than 2^8.
//
// In 8 bits the products run in fp16, which holds every code exactly and which a conversion
// instruction makes of two codes at once (putting codes into bf16 took more than half of the
// instructions; a product of changing 8-bit operands takes 53 cycles on this part's mma.sync, the two
// of 16 bits that replace it 16). A power
// of two per row brings Q's largest value to [2^14, 2^15), so that values down to 2^-28 of it keep
// bf16's 8 bits. The weights (softmax weight times the value's scale) have a factor of their own
// per row that keeps the largest at 2^6 or more and below 2^15, apart from the maximum that the
// row's sum is relative to: scales of any size keep 11 bits of every weight down to 2^-20 of the
// largest. O is in that frame. In bf16 the weights (2^8 at most) are held 2^-c down, a warp's sum at
// one or less, and O stays in range for values of any size (values below 2^(c - 126) lose bits: 2^-100).
// Warps' and CTAs' sums are joined as averages, for the same reason.
//
// The visible keys of all sequences and key heads form one list of chunks, cut evenly over
// the CTAs: sequences of different lengths balance, one long sequence fills the GPU. A CTA
// that holds a key head's whole list writes O itself; pieces go to the workspace (two slots per
// CTA) and attend_token_join_kernel adds them in order.
#pragma once

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

// Keys of a warp's step, and CTAs that fit an SM (registers: O^T, Q^T, K, V).
__host__ __device__ constexpr int token_keys(int d) { return 2048 / d; }
template <int D, bool E4M3, int NR>
__host__ __device__ constexpr int token_ctas_per_sm() {
  return NR == 2 ? (E4M3 ? 3 : 2) : (E4M3 ? 4 : 3);
}

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

// Joins the four warps' averages over chunks [c0, c1) of (b, hk), in warp order: rows of O if the CTA
// holds the whole list, a piece in the workspace if not.
template <int D, int NR>
__device__ __forceinline__ void join_warps(const AttendTokenParams& p, const TokenSight& s, int b, int hk, int c0, int c1,
                                           const float (&acc)[kTokenWarps][8 * NR][D + 4],
                                           const float (&stat)[2][kTokenWarps][8 * NR]) {
  const int G = p.Hq / p.Hkv, rows = s.nq * G;
  const bool all = c0 == 0 && c1 == s.chunks;
  const int64_t slot = 2 * int64_t(blockIdx.x) + (c0 == 0 ? 1 : 0);
  for (int e = threadIdx.x; e < rows * (D / 4); e += 32 * kTokenWarps) {
    const int r = e / (D / 4), d = e % (D / 4) * 4;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kTokenWarps; ++w) mm = fmaxf(mm, stat[0][w][r]);
    const float m0 = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f, part[kTokenWarps];
#pragma unroll
    for (int w = 0; w < kTokenWarps; ++w) {
      part[w] = tc::ex2(stat[0][w][r] - m0) * stat[1][w][r];  // a warp that saw nothing: 0, and its average is 0
      ll += part[w];
    }
    const float inv = ll != 0.f ? 1.f / ll : 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kTokenWarps; ++w) {
      const float4 y = *reinterpret_cast<const float4*>(&acc[w][r][d]);
      const float k = part[w] * inv;
      x.x = fmaf(k, y.x, x.x);
      x.y = fmaf(k, y.y, x.y);
      x.z = fmaf(k, y.z, x.z);
      x.w = fmaf(k, y.w, x.w);
    }
    const float lg = ll != 0.f ? m0 + __log2f(ll) : -INFINITY;
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

// D = A(16x16 fp16, row) * B(16x8 fp16, col) + D, fp32 accumulate.
__device__ __forceinline__ void mma_f16_16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 8 x 8 16-bit matrix, a row per four lanes, transposed across the warp
__device__ __forceinline__ uint32_t transpose8(uint32_t w) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(w));
  return r;
}

template <int D, bool E4M3, int NR>
__global__ void __launch_bounds__(32 * kTokenWarps, (token_ctas_per_sm<D, E4M3, NR>()))
attend_token_kernel(const AttendTokenParams p) {
  constexpr int KEYS = token_keys(D), NG = KEYS / 16, CHUNK = kTokenWarps * KEYS;
  constexpr int ROW = E4M3 ? D : 2 * D;  // bytes of a cache row
  constexpr int KCH = ROW / 64;          // 16-byte loads of a key per lane
  constexpr int VW = ROW / 32;           // words of a value per lane
  constexpr int MT = D / 16;             // products of 16 dimensions of O^T
  __shared__ float acc[kTokenWarps][8 * NR][D + 4];
  __shared__ float stat[2][kTokenWarps][8 * NR];
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
  const int page_mask = (1 << p.pages.log_page) - 1;
  const uint8_t* const baseK = static_cast<const uint8_t*>(p.pages.K);
  const uint8_t* const baseV = static_cast<const uint8_t*>(p.pages.V);

  while (u < end) {
    while (u >= before + (long long)s.chunks * p.Hkv) {  // sequences that see nothing have no chunks
      before += (long long)s.chunks * p.Hkv;
      s.set(p.pages, p.win, ++b, p.N, CHUNK);
    }
    const int hk = int((u - before) / s.chunks), c0 = int((u - before) % s.chunks);
    const int c1 = int(min((long long)s.chunks, c0 + (end - u)));
    const int rows = s.nq * G;
    // Q^T: the lane's column is row g (and 8 + g), the dimensions in the order of K's loads: 8 values
    // per 32 dimensions (bf16), 16 per 64 (8 bits)
    uint32_t qb[NR][D / 16][2];
    float up[NR];  // 8 bits: the power of two that Q's row took
#pragma unroll
    for (int h = 0; h < NR; ++h) {
      const int r = g + 8 * h;
      const bool real = r < rows;
      const int t = real ? r / G : 0, head = hk * G + (real ? r % G : 0);
      const bf16* src = p.Q + ((size_t(b) * p.Hq + head) * p.N + t) * D;
      uint4 w[D / 32];
      uint32_t top = 0;
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        const int d = E4M3 ? (x >> 1) * 64 + q * 16 + (x & 1) * 8 : x * 32 + q * 8;
        w[x] = real ? __ldg(reinterpret_cast<const uint4*>(src + d)) : make_uint4(0, 0, 0, 0);
        const uint32_t ww[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          qb[h][2 * x + (i >> 1)][i & 1] = ww[i];
          top = max(top, max(ww[i] & 0x7fffu, (ww[i] >> 16) & 0x7fffu));
        }
      }
      if constexpr (E4M3) {
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int field = min(253, 268 - int(top >> 7));  // top * 2^(field - 127) lies in [2^14, 2^15)
        const float f = top >= 0x7f80u ? __uint_as_float(0x7fc00000u) : exponent(field);  // infinity, NaN: NaN
        up[h] = exponent(254 - field);
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            qb[h][x][i] = pack_f16x2(bf16_lo(qb[h][x][i]) * f, bf16_hi(qb[h][x][i]) * f);
      }
    }
    // rows 8 h + 2 q + e: what they see, and the factor of their scores (base 2)
    int z[NR][2], a[NR][2];
    float sl2[NR][2];
#pragma unroll
    for (int h = 0; h < NR; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * h + 2 * q + e, t = r < rows ? r / G : 0;
        z[h][e] = max(-1, min(s.n - 1, s.n - s.nq + t + p.win.right));
        a[h][e] = max(0, s.n - s.nq + t - p.win.left);
        sl2[h][e] = p.scale * 1.4426950408889634f;
        if constexpr (E4M3) sl2[h][e] *= __shfl_sync(0xffffffffu, up[h], (2 * q + e) * 4);
      }
    constexpr int kTopField = 247;  // the weights' factor f is at most 2^120
    const int down = 40 - __clz(max(c1 - c0, 1) * KEYS - 1);  // bf16: c, the weights of a warp's keys sum to 2^c at most
    const float frame = exponent(127 - down);
    float o[NR][MT][4], m[NR][2], l[NR][2], f[NR][2];
#pragma unroll
    for (int h = 0; h < NR; ++h) {
#pragma unroll
      for (int i = 0; i < MT; ++i) o[h][i][0] = o[h][i][1] = o[h][i][2] = o[h][i][3] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[h][e] = -INFINITY;
        l[h][e] = 0.f;
        f[h][e] = exponent(kTopField);
      }
    }

    uint4 kr[NG][2][KCH];
    uint32_t vr[NG][4][VW];
    float ks[NG][2], vs[NG][2];  // scales of keys g and 8 + g
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
        const int64_t row = ((int64_t(page) * p.Hkv + hk) << p.pages.log_page) + (j & page_mask) + g;
        const uint8_t* src = baseK + row * ROW + q * 16;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const bool ok = all || (page >= 0 && in(j + 8 * t + g));
#pragma unroll
          for (int x = 0; x < KCH; ++x) {
            if constexpr (all) kr[i][t][x] = ldg_stream_v4(src + 8 * t * ROW + x * 64);
            else kr[i][t][x] = ldg16(src + 8 * t * ROW + x * 64, ok);
          }
          if constexpr (E4M3) ks[i][t] = ok ? __ldg(p.pages.ks + row + 8 * t) : 0.f;
        }
      }
    };
    auto load_v = [&](int c, int held, auto all) {
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        const int page = __shfl_sync(0xffffffffu, held, i), j = s.key(c, CHUNK) + warp * KEYS + i * 16;
        const int64_t row = ((int64_t(page) * p.Hkv + hk) << p.pages.log_page) + (j & page_mask);
        // 16 bytes per lane and 128 (a 64-byte row: 8 bytes)
        const uint8_t* src = baseV + (row + 2 * q) * ROW + g * (ROW < 128 ? 8 : 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // keys 2q, 2q + 1, 2q + 8, 2q + 9
          const int key = (e & 1) + (e >> 1) * 8;
          const bool ok = all || (page >= 0 && in(j + 2 * q + key));
          if constexpr (ROW < 128) {
            const uint2 w = ok ? __ldg(reinterpret_cast<const uint2*>(src + key * ROW)) : make_uint2(0, 0);
            vr[i][e][0] = w.x;
            vr[i][e][1] = w.y;
          } else {
#pragma unroll
            for (int x = 0; x < VW / 4; ++x) {
              uint4 w;
              if constexpr (all) w = ldg_stream_v4(src + key * ROW + x * 128);
              else w = ldg16(src + key * ROW + x * 128, ok);
              vr[i][e][4 * x] = w.x;
              vr[i][e][4 * x + 1] = w.y;
              vr[i][e][4 * x + 2] = w.z;
              vr[i][e][4 * x + 3] = w.w;
            }
          }
        }
        if constexpr (E4M3) {
#pragma unroll
          for (int t = 0; t < 2; ++t)
            vs[i][t] = all || (page >= 0 && in(j + 8 * t + g)) ? __ldg(p.pages.vs + row + g + 8 * t) : 0.f;
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
    // maximum over the lanes of the same rows
    auto over_keys = [](float x) {
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
      return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
    };
    int held = pages_of(c0);
    bool all = full(c0, held);
    fetch_k(c0, held, all);
    fetch_v(c0, held, all);
    int next = pages_of(c0 + 1);
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
      const int j0 = s.key(c, CHUNK) + warp * KEYS;
      // S^T: element e + 2 t of product (i, h): key 16 i + 8 t + g, row 8 h + 2 q + e
      float sc[NG][NR][4];
#pragma unroll
      for (int i = 0; i < NG; ++i) {
#pragma unroll
        for (int h = 0; h < NR; ++h) sc[i][h][0] = sc[i][h][1] = sc[i][h][2] = sc[i][h][3] = 0.f;
#pragma unroll
        for (int x = 0; x < KCH; ++x) {
          const uint32_t w0[4] = {kr[i][0][x].x, kr[i][0][x].y, kr[i][0][x].z, kr[i][0][x].w};
          const uint32_t w1[4] = {kr[i][1][x].x, kr[i][1][x].y, kr[i][1][x].z, kr[i][1][x].w};
          if constexpr (E4M3) {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              const uint32_t ka[4] = {codes_to_f16_lo(w0[y]), codes_to_f16_lo(w1[y]), codes_to_f16_hi(w0[y]), codes_to_f16_hi(w1[y])};
#pragma unroll
              for (int h = 0; h < NR; ++h) mma_f16_16816(sc[i][h], ka, qb[h][4 * x + y][0], qb[h][4 * x + y][1]);
            }
          } else {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t ka[4] = {w0[2 * y], w1[2 * y], w0[2 * y + 1], w1[2 * y + 1]};
#pragma unroll
              for (int h = 0; h < NR; ++h) mma_bf16_16816(sc[i][h], ka, qb[h][2 * x + y][0], qb[h][2 * x + y][1]);
            }
          }
        }
        if constexpr (E4M3) {
#pragma unroll
          for (int h = 0; h < NR; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[i][h][e] *= ks[i][e >> 1];
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
          for (int h = 0; h < NR; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = j0 + i * 16 + 8 * (e >> 1) + g;
              if (!(here && j <= z[h][e & 1] && (j >= a[h][e & 1] || j < p.win.sinks))) sc[i][h][e] = -INFINITY;
            }
        }
      }
      bool grow = false;
      float mx[NR][2];
#pragma unroll
      for (int h = 0; h < NR; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[h][e] = fmaxf(sc[0][h][e], sc[0][h][e + 2]);
#pragma unroll
          for (int i = 1; i < NG; ++i) mx[h][e] = fmaxf(mx[h][e], fmaxf(sc[i][h][e], sc[i][h][e + 2]));
          mx[h][e] *= sl2[h][e];
          grow |= mx[h][e] > m[h][e] + 8.f;
        }
      if (__any_sync(0xffffffffu, grow)) {  // the sums follow the maximum in steps of 2^8 or more
#pragma unroll
        for (int h = 0; h < NR; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float top = over_keys(mx[h][e]);
            if (!(top > m[h][e] + 8.f)) continue;
            if (m[h][e] != -INFINITY) {
              const float k = tc::ex2(m[h][e] - top);
              l[h][e] *= k;
              if constexpr (E4M3) {  // O stays, its frame's factor grows (and is bounded below)
                f[h][e] *= tc::ex2(top - m[h][e]);
              } else {
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                  o[h][i][e] *= k;
                  o[h][i][e + 2] *= k;
                }
              }
            }
            m[h][e] = top;
          }
      }
      // Tokens that do not all see the step: a value that is no finite number would reach them through
      // a weight of zero. It leaves the products, and joins O of the rows that see it here.
      if (!whole && s.see.p0 != s.see.p1) {
        auto sees = [&](int j, int h, int e) { return j <= z[h][e] && (j >= a[h][e] || j < p.win.sinks); };
        bool odd = false;
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          if constexpr (E4M3) {
            odd |= !(fabsf(vs[i][0]) < INFINITY) || !(fabsf(vs[i][1]) < INFINITY);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
              for (int x = 0; x < VW; x += 4)
                odd |= any_not_finite(make_uint4(vr[i][e][x], vr[i][e][x + 1], vr[i][e][x + 2], vr[i][e][x + 3]));
          }
        }
        if (__any_sync(0xffffffffu, odd)) {
#pragma unroll
          for (int i = 0; i < NG; ++i) {
            if constexpr (E4M3) {  // NaN in every column
#pragma unroll
              for (int t = 0; t < 2; ++t) {
                const bool bad = !(fabsf(vs[i][t]) < INFINITY);
                if (bad) vs[i][t] = 0.f;
                // its codes may be NaN too: those of keys 2 q and 2 q + 1 (and 8 more) are this lane's,
                // their scales lanes 8 q's and 8 q + 4's
                const uint32_t rows = __ballot_sync(0xffffffffu, bad);
#pragma unroll
                for (int e2 = 0; e2 < 2; ++e2)
                  if ((rows >> (8 * q + 4 * e2)) & 1u)
#pragma unroll
                    for (int x = 0; x < VW; ++x) vr[i][2 * t + e2][x] = 0u;
#pragma unroll
                for (int h = 0; h < NR; ++h)
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    const uint32_t lanes = __ballot_sync(0xffffffffu, bad && sees(j0 + i * 16 + 8 * t + g, h, e));
                    if (!(lanes & (0x11111111u << q))) continue;
#pragma unroll
                    for (int x = 0; x < MT; ++x) o[h][x][e] = o[h][x][e + 2] = __uint_as_float(0x7fc00000u);
                  }
              }
            } else {
#pragma unroll 1
              for (int from = 0; from < 4; ++from)  // the lanes of the quad hold four keys each
#pragma unroll
                for (int e4 = 0; e4 < 4; ++e4)
#pragma unroll
                  for (int x = 0; x < VW; ++x) {
                    const uint32_t v = __shfl_sync(0xffffffffu, vr[i][e4][x], (lane & ~3) + from);
                    const int j = j0 + i * 16 + 2 * from + (e4 & 1) + (e4 >> 1) * 8;
#pragma unroll
                    for (int h = 0; h < NR; ++h)
#pragma unroll
                      for (int e = 0; e < 2; ++e)
                        if (sees(j, h, e)) {
                          o[h][x][e] += not_finite_lo(v);
                          o[h][x][e + 2] += not_finite_hi(v);
                        }
                  }
#pragma unroll
              for (int e4 = 0; e4 < 4; ++e4)
#pragma unroll
                for (int x = 0; x < VW; ++x) vr[i][e4][x] = finite_or_zero(vr[i][e4][x]);
            }
          }
        }
      }
      bool wide = false;
      float tm[NR][2];
#pragma unroll
      for (int h = 0; h < NR; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float neg = m[h][e] == -INFINITY ? 0.f : -m[h][e];
          tm[h][e] = 0.f;
#pragma unroll
          for (int i = 0; i < NG; ++i)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const float w = tc::ex2(fmaf(sc[i][h][e + 2 * t], sl2[h][e], neg));
              l[h][e] += w;
              sc[i][h][e + 2 * t] = w * (E4M3 ? vs[i][t] : frame);
              if constexpr (E4M3) tm[h][e] = fmaxf(tm[h][e], sc[i][h][e + 2 * t]);
            }
          if constexpr (E4M3) wide |= f[h][e] > exponent(kTopField) || tm[h][e] * f[h][e] > 32768.f;
        }
      if constexpr (E4M3) {
        if (__any_sync(0xffffffffu, wide)) {
#pragma unroll
          for (int h = 0; h < NR; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float top = over_keys(tm[h][e]), old = f[h][e];
              // the largest weight passes 2^15: bring it to [2^6, 2^7)
              if (top * old > 32768.f) f[h][e] = exponent(min(kTopField, 260 - int(__float_as_uint(top) >> 23)));
              else f[h][e] = fminf(old, exponent(kTopField));
              // a factor past 2^122 (infinity too): what O holds is too small to count
              const float k = f[h][e] == old ? 1.f : (old > 5e36f ? 0.f : __fdividef(f[h][e], old));
#pragma unroll
              for (int i = 0; i < MT; ++i) {
                o[h][i][e] *= k;
                o[h][i][e + 2] *= k;
              }
            }
        }
      }
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        uint32_t pb[NR][2];  // P^T: keys 2 q, 2 q + 1 (and 8 more) of row g
#pragma unroll
        for (int h = 0; h < NR; ++h)
#pragma unroll
          for (int t = 0; t < 2; ++t)
            pb[h][t] = transpose8(E4M3 ? pack_f16x2(sc[i][h][2 * t] * f[h][0], sc[i][h][2 * t + 1] * f[h][1])
                                       : pack_bf16x2(sc[i][h][2 * t], sc[i][h][2 * t + 1]));
        // O^T: word x of the lane's values gives dimensions d0 and d0 + 1 (bf16), or two such pairs
#pragma unroll
        for (int x = 0; x < VW; ++x) {
          const uint32_t v0 = vr[i][0][x], v1 = vr[i][1][x], v2 = vr[i][2][x], v3 = vr[i][3][x];
          if constexpr (E4M3) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t lo = __byte_perm(v0, v1, y ? 0x7362 : 0x5140), hi = __byte_perm(v2, v3, y ? 0x7362 : 0x5140);
              const uint32_t va[4] = {codes_to_f16_lo(lo), codes_to_f16_hi(lo), codes_to_f16_lo(hi), codes_to_f16_hi(hi)};
#pragma unroll
              for (int h = 0; h < NR; ++h) mma_f16_16816(o[h][2 * x + y], va, pb[h][0], pb[h][1]);
            }
          } else {
            const uint32_t va[4] = {__byte_perm(v0, v1, 0x5410), __byte_perm(v0, v1, 0x7632), __byte_perm(v2, v3, 0x5410),
                                    __byte_perm(v2, v3, 0x7632)};
#pragma unroll
            for (int h = 0; h < NR; ++h) mma_bf16_16816(o[h][x], va, pb[h][0], pb[h][1]);
          }
        }
      }
      if (c + 1 < c1) fetch_v(c + 1, next, next_all);
      held = next;
      all = next_all;
      next = pages_of(c + 2);
    }
    // the warps' accumulators, joined in warp order
    __syncthreads();  // the previous key head's joined rows have been read
#pragma unroll
    for (int h = 0; h < NR; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * h + 2 * q + e;
        const float k = E4M3 ? 1.f / f[h][e] : exponent(127 + down);
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[h][e] += __shfl_xor_sync(0xffffffffu, l[h][e], off);
        const float inv = l[h][e] != 0.f ? 1.f / l[h][e] : 0.f;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          // rows g and 8 + g of product i are neighbouring dimensions
          const int d = E4M3 ? g * (D / 8) + 2 * i : (i >> 2) * 64 + g * 8 + 2 * (i & 3);
          *reinterpret_cast<float2*>(&acc[warp][r][d]) = make_float2(o[h][i][e] * inv * k, o[h][i][e + 2] * inv * k);
        }
        if (g == 0) {
          stat[0][warp][r] = m[h][e];
          stat[1][warp][r] = l[h][e];
        }
      }
    __syncthreads();
    join_warps<D, NR>(p, s, b, hk, c0, c1, acc, stat);
    u += c1 - c0;
  }
}

// One block per row: joins the pieces that several CTAs hold and writes the rows of sequences
// that see nothing. The block's D/4 lanes of columns times its groups of pieces; the groups' sums
// are added in order.
template <int D>
__global__ void __launch_bounds__(32 * kTokenWarps) attend_token_join_kernel(const AttendTokenParams p) {
  constexpr int CHUNK = kTokenWarps * token_keys(D), LANES = D / 4, GROUPS = 32 * kTokenWarps / LANES;
  __shared__ long long sh[kTokenWarps + 2];
  __shared__ float top[kTokenWarps];
  __shared__ float4 part[GROUPS][LANES];
  __shared__ float sum[GROUPS];
  const int G = p.Hq / p.Hkv, R = G * p.N;
  const int b = blockIdx.x / (p.Hkv * R), hk = blockIdx.x / R % p.Hkv, r = blockIdx.x % R;
  const UnitAt at = find_unit<CHUNK>(p, b, 0, sh);
  TokenSight s;
  s.set(p.pages, p.win, b, p.N, CHUNK);
  const long long u0 = at.before + (long long)hk * s.chunks, u1 = u0 + s.chunks;
  // the CTA that holds unit u is the last one whose first unit is not behind it
  const int first = s.chunks ? int(((u0 + 1) * at.ctas - 1) / at.total) : 0;
  const int last = s.chunks ? int((u1 * at.ctas - 1) / at.total) : -1;
  // every block waits, so that this grid does not end before the one it depends on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (first == last || r >= s.nq * G) return;
  auto slot = [&](int c) { return (2 * int64_t(c) + (c == first)) * kTokenRows + r; };
  float m = -INFINITY;
  for (int c = first + int(threadIdx.x); c <= last; c += blockDim.x) m = fmaxf(m, p.part_lse[slot(c)]);
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kTokenWarps; ++w) m = fmaxf(m, top[w]);
  const float m0 = m == -INFINITY ? 0.f : m;
  const int col = threadIdx.x % LANES, group = threadIdx.x / LANES;
  float l = 0.f;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int c = first + group; c <= last; c += GROUPS) {
    const float w = tc::ex2(p.part_lse[slot(c)] - m0) * exponent(127 - 10);  // no more than 592 pieces: in range
    const float4 y = *reinterpret_cast<const float4*>(p.part + slot(c) * D + col * 4);
    l += w;
    x.x = fmaf(w, y.x, x.x);
    x.y = fmaf(w, y.y, x.y);
    x.z = fmaf(w, y.z, x.z);
    x.w = fmaf(w, y.w, x.w);
  }
  part[group][col] = x;
  if (col == 0) sum[group] = l;
  __syncthreads();
  if (group != 0) return;
#pragma unroll
  for (int i = 1; i < GROUPS; ++i) {
    const float4 y = part[i][col];
    l += sum[i];
    x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  const size_t row = (size_t(b) * p.Hq + hk * G + r % G) * p.N + r / G;
  *reinterpret_cast<uint2*>(p.O + row * D + col * 4) = make_uint2(pack_bf16x2(x.x * inv, x.y * inv), pack_bf16x2(x.z * inv, x.w * inv));
  if (col == 0 && p.lse) p.lse[row] = l != 0.f ? (m0 + __log2f(l * exponent(127 + 10))) * 0.6931471805599453f : -INFINITY;
}

}  // namespace pisa
