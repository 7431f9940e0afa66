// Gradient of the windowed attention on the tensor cores (tcgen05 / TMEM / TMA).
//
//   p = exp(s - lse),  delta = do.o,  dp = do.v,  ds = p (dp - delta)
//   dq = scale sum_j ds k_j      dk_j = scale sum ds q,  dv_j = sum p do
//
// With lse known no row statistic is left to find, so the weights of a tile are computed
// independently, by two threads or two groups of threads at once. Two kernels compute the
// scores anew rather than add dQ up with atomics: their sums run in a fixed order.
//
// attend_dq_kernel: a CTA takes a row tile of a key head (as the forward kernel's) and walks the key
// tiles that it sees. Tensor memory:
// dQ (D columns), S in two buffers and dP in one (128 columns each); dS in bf16 overwrites
// its S. Tile i + 1's S and (as soon as the row threads hold dP(i) in registers) dP are
// issued before dS(i) is awaited, so the weights are computed under the products. It also
// writes delta for the other kernel.
//
// attend_dkv_kernel: a CTA takes 128 keys and walks 64-row tiles of the queries that see
// them, head by head, with the scores transposed (lane = key): S^T = K Q^T and dP^T = V dO^T
// into one of two buffers, then dV += P^T dO and dK += dS^T Q with P^T and dS^T from tensor
// memory. Two groups of four warps take alternate tiles. A key tile that many rows see (the
// first tokens, or a causal sequence's) is cut into runs; their fp32 partial sums are joined
// in run order by attend_dkv_join_kernel.
//
// Bound: tensor time. Per 128 x 128 scores at D = 128, dQ: three products of 512 cycles;
// dK, dV: 64-column products take 48 cycles per 16 dimensions, not 32, so 2 x 2 x 390 for
// S^T and dP^T and 2 x 2 x 256 for dV and dK. 128-row tiles would leave tensor memory no
// second buffer, and the weights would wait on the products.
// Measured on 16384 tokens, 16 query and 4 key heads of 128, causal over 2048 keys: dQ 366 us (1.09
// PFLOP/s of its 6 d flops per pair and query head; 500 us with strided loads of the rows and one
// ring for K and V), dK and dV 547 us (0.97 of its 8 d), the join 11 us. What they wait for is each
// other: the hand-offs between products and weights. A third buffer would hide them; at D = 128 tensor
// memory has no room for one (at D = 64, where dV, dK and two buffers take 384 columns, it has: not
// built). Cutting the runs by a model of their cost instead of evenly: 2% slower.
// The dK, dV kernel and the join set up while the kernel before them ends: a step on 2049 tokens,
// 12 and 4 heads of 64, takes 67 us with that and 71 without.
#pragma once

#include "attend_tc.cuh"

namespace pisa {

struct AttendGradParams {
  const bf16* Q;
  const bf16* O;
  const bf16* dO;
  const float* lse;
  float* delta;
  bf16 *dQ, *dK, *dV;
  float* part;  // runs of split key tiles: fp32 [slot][dV, dK][128][D]
  int B, Hq, Hkv, N;
  RowTiles rt;
  Window win;
  float scale;
  int run;      // query tiles per run, at most
  int runs;     // runs of a key head
  int slots;    // partial sums of a key head
};

// ------------------------------------------------------------------ dQ
template <int D>
struct AttendDqCfg {
  static constexpr int kThreads = 384;
  static constexpr int TILE = 128 * D * 2;
  // K is held from its scores to its dQ product, V only for dP: rings of their own, so that V of the
  // next tile does not queue behind K of the last
  static constexpr int NK = D == 128 ? 3 : 5, NV = D == 128 ? 2 : 4;
  static constexpr int OFF_Q = 0, OFF_DO = TILE, OFF_K = 2 * TILE, OFF_V = OFF_K + NK * TILE;
  static constexpr int OFF_X = OFF_V + NV * TILE;  // float [2][128]: halves of delta
  static constexpr int OFF_BAR = OFF_X + 1024;
  static constexpr int B_KFULL = 0, B_KEMPTY = B_KFULL + NK, B_VFULL = B_KEMPTY + NK, B_VEMPTY = B_VFULL + NV;
  static constexpr int B_Q = B_VEMPTY + NV;  // Q, dO and O (in the last V stage) landed
  static constexpr int B_X = B_Q + 1;        // delta computed: that stage is V's (8 warps)
  static constexpr int B_SD = B_X + 1;   // S and dP ready (commit)
  static constexpr int B_R = B_SD + 1;   // dP read (8 warps)
  static constexpr int B_DS = B_R + 1;   // dS written (8 warps)
  static constexpr int B_O = B_DS + 1;   // all products done (commit)
  static constexpr int NBARS = B_O + 1;
  static constexpr int OFF_MISC = OFF_BAR + 8 * NBARS;
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
  static constexpr int DQ_COL = 0, S_COL = 128, DP_COL = 384;
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

template <int D>
__global__ void __launch_bounds__(384, 1)
attend_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmG,
                 const __grid_constant__ CUtensorMap tmO, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, const AttendGradParams p) {
  using C = AttendDqCfg<D>;
  using namespace tc;
  extern __shared__ __align__(16) uint8_t attend_dq_smem[];
  const uint32_t raw_u = smem_u32(attend_dq_smem);
  const uint32_t base_u = (raw_u + 1023u) & ~1023u;
  uint8_t* base = attend_dq_smem + (base_u - raw_u);
  volatile int* abort_flag = reinterpret_cast<int*>(base + C::OFF_MISC) + 1;
  const uint32_t bar0 = base_u + C::OFF_BAR;
  asm volatile("griddepcontrol.launch_dependents;");
#define ABAR(i) (bar0 + 8u * uint32_t(i))
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const int G = p.Hq / p.Hkv, tokens = p.rt.tokens;
  const int part_tiles = (p.N + tokens - 1) / tokens, row_tiles = part_tiles * p.rt.parts;
  const int bh = blockIdx.x / row_tiles, tile = blockIdx.x - bh * row_tiles, part = tile / part_tiles;
  const int t0 = (part_tiles - 1 - (tile - part * part_tiles)) * tokens;  // causal: the rows with the most keys first
  const int head0 = bh * G + part * 128, heads = min(p.rt.heads, G - part * 128);
  Sight see;
  see.set(p.win, t0, min(t0 + tokens, p.N) - 1, p.N);
  TileList tiles;
  tiles.set(see, 0, 1);
  const int count = tiles.to;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NK; ++s) {
      mbar_init(ABAR(C::B_KFULL + s), 1);
      mbar_init(ABAR(C::B_KEMPTY + s), 1);
    }
    for (int s = 0; s < C::NV; ++s) {
      mbar_init(ABAR(C::B_VFULL + s), 1);
      mbar_init(ABAR(C::B_VEMPTY + s), 1);
    }
    mbar_init(ABAR(C::B_Q), 1);
    mbar_init(ABAR(C::B_X), 8);
    mbar_init(ABAR(C::B_SD), 1);
    mbar_init(ABAR(C::B_R), 8);
    mbar_init(ABAR(C::B_DS), 8);
    mbar_init(ABAR(C::B_O), 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 2) {
    tmem_alloc(base_u + C::OFF_MISC, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<uint32_t*>(base + C::OFF_MISC);

  if (warp == 0) {
    // lanes 0 and 1: the two 64-column panels
    if (lane < 2) {
      bool ok = true;
      const uint32_t bytes = uint32_t(tokens * p.rt.heads * D * 2);
      if (lane == 0) mbar_arrive_expect_tx(ABAR(C::B_Q), 3 * bytes);
      __syncwarp(0x3u);
      if (lane * 64 < D) {
        tma_load_3d(base_u + C::OFF_Q + lane * 16384, &tmQ, ABAR(C::B_Q), lane * 64, t0, head0);
        tma_load_3d(base_u + C::OFF_DO + lane * 16384, &tmG, ABAR(C::B_Q), lane * 64, t0, head0);
        tma_load_3d(base_u + C::OFF_V + (C::NV - 1) * C::TILE + lane * 16384, &tmO, ABAR(C::B_Q), lane * 64, t0, head0);
      }
      int i = 0, v_used = 0;
      for (; i < count && ok; ++i) {
        const int sk = i % C::NK, sv = i % C::NV;
        ok = __all_sync(0x3u, wait_bounded(ABAR(C::B_KEMPTY + sk), ((i / C::NK) & 1) ^ 1, abort_flag));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(ABAR(C::B_KFULL + sk), C::TILE);
        __syncwarp(0x3u);
        if (lane * 64 < D)
          tma_load_3d(base_u + C::OFF_K + sk * C::TILE + lane * 16384, &tmK, ABAR(C::B_KFULL + sk), lane * 64, tiles.key(i), bh);
        if (i == C::NV - 1) ok = wait_bounded(ABAR(C::B_X), 0, abort_flag);  // O has been read
        ok = __all_sync(0x3u, ok && wait_bounded(ABAR(C::B_VEMPTY + sv), ((i / C::NV) & 1) ^ 1, abort_flag));
        if (!ok) {
          ++i;  // this tile's K is in flight
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(ABAR(C::B_VFULL + sv), C::TILE);
        __syncwarp(0x3u);
        if (lane * 64 < D)
          tma_load_3d(base_u + C::OFF_V + sv * C::TILE + lane * 16384, &tmV, ABAR(C::B_VFULL + sv), lane * 64, tiles.key(i), bh);
        v_used = i + 1;
      }
      // no copy may still be in flight when the CTA exits
      if (lane == 0) {
        wait_drain(ABAR(C::B_Q), 0);
        for (int u = i > C::NK ? i - C::NK : 0; u < i; ++u) wait_drain(ABAR(C::B_KFULL + u % C::NK), (u / C::NK) & 1);
        for (int u = v_used > C::NV ? v_used - C::NV : 0; u < v_used; ++u) wait_drain(ABAR(C::B_VFULL + u % C::NV), (u / C::NV) & 1);
      }
    }
  } else if (warp == 1) {
    constexpr uint32_t idS = idesc_bf16(128, 128, false), idQ = idesc_bf16(128, D, true);
    const bool lead = elect();
    auto rows_by = [&](uint32_t a, uint32_t t, uint32_t col) {  // A [128 rows][D] times the tile, transposed
      const uint64_t da = operand(a, 16), dt = operand(t, 16);
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        const uint32_t off = ((c >> 2) * 16384 + (c & 3) * 32) >> 4;
        umma_ss(tmem + col, da + off, dt + off, idS, c ? 1u : 0u);
      }
    };
    bool ok = wait_warp(ABAR(C::B_Q), 0, abort_flag);
    for (int i = -1; i < count && ok; ++i) {
      const int n = i + 1;
      if (n < count) {
        if (!(ok = wait_warp(ABAR(C::B_KFULL + n % C::NK), (n / C::NK) & 1, abort_flag))) break;
        tc_fence_after();
        if (lead) rows_by(base_u + C::OFF_Q, base_u + C::OFF_K + (n % C::NK) * C::TILE, C::S_COL + (n & 1) * 128);
        if (i >= 0 && !(ok = wait_warp(ABAR(C::B_R), i & 1, abort_flag))) break;
        if (!(ok = wait_warp(ABAR(C::B_VFULL + n % C::NV), (n / C::NV) & 1, abort_flag))) break;
        tc_fence_after();
        if (lead) {
          rows_by(base_u + C::OFF_DO, base_u + C::OFF_V + (n % C::NV) * C::TILE, C::DP_COL);
          umma_commit(ABAR(C::B_SD));
          umma_commit(ABAR(C::B_VEMPTY + n % C::NV));
        }
      }
      if (i < 0) continue;
      if (!(ok = wait_warp(ABAR(C::B_DS), i & 1, abort_flag))) break;
      tc_fence_after();
      if (lead) {
        const uint64_t k = operand(base_u + C::OFF_K + (i % C::NK) * C::TILE, 16384);
        const uint32_t ds = tmem + C::S_COL + (i & 1) * 128;
        // keys [16c, 16c + 16): the thread of half c / 4 packed them at the start of its columns
#pragma unroll
        for (int c = 0; c < 8; ++c)
          umma_ts(tmem + C::DQ_COL, ds + (c >> 2) * 64 + (c & 3) * 8, k + c * (2048 >> 4), idQ, (i | c) ? 1u : 0u);
        umma_commit(ABAR(C::B_KEMPTY + i % C::NK));
      }
    }
    if (lead) {
      umma_commit(ABAR(C::B_O));
      wait_drain(ABAR(C::B_O), 0);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // two threads per row: half hf has keys [64 hf, 64 hf + 64) of a tile, and D/2 dimensions
    const int hf = (warp - 4) >> 2, rt = threadIdx.x & 127;
    const int my_head = rt / tokens, my_token = rt - my_head * tokens;
    const bool real = my_head < heads && t0 + my_token < p.N;
    const int t = t0 + (real ? my_token : 0);
    const size_t row = size_t(head0 + (real ? my_head : 0)) * p.N + t;
    const uint32_t lrow = uint32_t((warp & 3) * 32) << 16;
    bool ok = __all_sync(0xffffffffu, wait_bounded(ABAR(C::B_Q), 0, abort_flag));
    float delta = 0.f;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      const int ch = hf * (D / 16) + c;
      const uint32_t off = (ch >> 3) * 16384 + rt * 128 + (((ch & 7) ^ (rt & 7)) << 4);
      const uint4 y = *reinterpret_cast<const uint4*>(base + C::OFF_DO + off);
      const uint4 w = *reinterpret_cast<const uint4*>(base + C::OFF_V + (C::NV - 1) * C::TILE + off);
      const uint32_t a[4] = {y.x, y.y, y.z, y.w}, e[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        delta = fmaf(bf16_lo(a[k]), bf16_lo(e[k]), delta);
        delta = fmaf(bf16_hi(a[k]), bf16_hi(e[k]), delta);
      }
    }
    fence_proxy_async_smem();  // reads of O before V's copies into its stage
    warp_arrive(ABAR(C::B_X));
    float* xd = reinterpret_cast<float*>(base + C::OFF_X);
    xd[hf * 128 + rt] = delta;
    ok = pair_sync_and(1 + (warp & 3), ok);
    delta = xd[rt] + xd[128 + rt];  // the same order on both sides
    if (real && hf == 0) p.delta[row] = delta;
    const float lse2 = real ? p.lse[row] * 1.4426950408889634f : 0.f, sl2 = p.scale * 1.4426950408889634f;
    const int z = min(p.N - 1, t + p.win.right), a = max(0, t - p.win.left);
    for (int i = 0; i < count && ok; ++i) {
      const int j0 = tiles.key(i) + hf * 64;
      const bool whole = j0 + 63 <= see.p0 + p.win.right && j0 + 64 <= p.N &&
                         (j0 >= see.p1 - p.win.left || j0 + 64 <= p.win.sinks);
      ok = __all_sync(0xffffffffu, wait_bounded(ABAR(C::B_SD), i & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      const uint32_t sa = tmem + lrow + C::S_COL + (i & 1) * 128 + hf * 64;
      uint32_t dp[64], sc[64];
#pragma unroll
      for (int ch = 0; ch < 4; ++ch)
        tmem_ld16(tmem + lrow + C::DP_COL + hf * 64 + ch * 16, *reinterpret_cast<uint32_t(*)[16]>(&dp[ch * 16]));
#pragma unroll
      for (int ch = 0; ch < 4; ++ch) tmem_ld16(sa + ch * 16, *reinterpret_cast<uint32_t(*)[16]>(&sc[ch * 16]));
#pragma unroll
      for (int ch = 0; ch < 4; ++ch) {
        tmem_wait_ld(*reinterpret_cast<uint32_t(*)[16]>(&dp[ch * 16]));
        tmem_wait_ld(*reinterpret_cast<uint32_t(*)[16]>(&sc[ch * 16]));
      }
      tc_fence_before();
      warp_arrive(ABAR(C::B_R));
#pragma unroll
      for (int k = 0; k < 64; k += 2) {
        float e0 = __uint_as_float(sc[k]), e1 = __uint_as_float(sc[k + 1]);
        fma2(e0, e1, sl2, -lse2);
        sc[k] = __float_as_uint(ex2(e0) * (__uint_as_float(dp[k]) - delta));
        sc[k + 1] = __float_as_uint(ex2(e1) * (__uint_as_float(dp[k + 1]) - delta));
      }
      if (!whole) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint32_t bits = ones_below(z - j0 + 1 - 32 * w) &
                                (~ones_below(a - j0 - 32 * w) | ones_below(p.win.sinks - j0 - 32 * w));
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (!((bits >> k) & 1u)) sc[32 * w + k] = 0u;
        }
      }
#pragma unroll
      for (int ch = 0; ch < 2; ++ch) {
        uint32_t pk[16];
#pragma unroll
        for (int k = 0; k < 16; ++k)
          pk[k] = pack_bf16x2(__uint_as_float(sc[ch * 32 + 2 * k]), __uint_as_float(sc[ch * 32 + 2 * k + 1]));
        tmem_st16(sa + ch * 16, pk);
      }
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(ABAR(C::B_DS));
    }
    ok = __all_sync(0xffffffffu, ok && wait_bounded(ABAR(C::B_O), 0, abort_flag));
    tc_fence_after();
#pragma unroll 1
    for (int ch = 0; ch < D / 64; ++ch) {
      __syncwarp();
      uint32_t x[2][16];
      const int c0 = hf * (D / 2) + ch * 32;
      tmem_ld16(tmem + lrow + C::DQ_COL + c0, x[0]);
      tmem_ld16(tmem + lrow + C::DQ_COL + c0 + 16, x[1]);
      tmem_wait_ld(x[0]);
      tmem_wait_ld(x[1]);
      store_rows32(p.dQ + c0, real && ok ? int64_t(row) * D : -1, x, p.scale);
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
#undef ABAR
}

// ------------------------------------------------------------------ dK, dV

// The 64-row query tiles [first, first + count) that see some key of tile kt.
struct QueryRange {
  int first, count;
  __host__ __device__ QueryRange(const Window& w, int kt, int N) {
    const int j0 = kt * 128, j1 = (j0 + 127 < N ? j0 + 127 : N - 1);
    const int lo = j0 > w.right ? j0 - w.right : 0;
    const long long far = (long long)j1 + w.left;
    const int hi = j0 < w.sinks || far > N - 1 ? N - 1 : int(far);
    first = lo / 64;
    count = hi / 64 - first + 1;
  }
};
__host__ __device__ inline int query_runs(int tiles, int run) { return (tiles + run - 1) / run; }

// Finds run `at` of a key head among its key tiles, or (kt given) a key tile's first slot.
// One warp; every lane gets the result.
struct RunAt {
  int kt, run, runs, slot;
};
__device__ __forceinline__ RunAt find_run(const AttendGradParams& p, int at, int want_kt) {
  const int lane = threadIdx.x & 31, G = p.Hq / p.Hkv, kts = (p.N + 127) / 128;
  int before = 0, slots = 0;
  for (int k0 = 0; k0 < kts; k0 += 32) {
    const int kt = k0 + lane;
    int r = 0;
    if (kt < kts) r = query_runs(G * QueryRange(p.win, kt, p.N).count, p.run);
    int x = r, y = r > 1 ? r : 0;
    const int mine = y;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, x, off), c = __shfl_up_sync(0xffffffffu, y, off);
      if (lane >= off) {
        x += a;
        y += c;
      }
    }
    const bool hit = kt < kts && (want_kt >= 0 ? kt == want_kt : (at >= before + x - r && at < before + x));
    const unsigned who = __ballot_sync(0xffffffffu, hit);
    if (who) {
      const int src = __ffs(who) - 1;
      RunAt f;
      f.kt = k0 + src;
      f.runs = __shfl_sync(0xffffffffu, r, src);
      f.run = at - before - (__shfl_sync(0xffffffffu, x, src) - f.runs);
      f.slot = slots + __shfl_sync(0xffffffffu, y - mine, src);
      return f;
    }
    before += __shfl_sync(0xffffffffu, x, 31);
    slots += __shfl_sync(0xffffffffu, y, 31);
  }
  return RunAt{0, 0, 0, 0};
}

template <int D>
struct AttendDkvCfg {
  static constexpr int kThreads = 384;
  static constexpr int KTILE = 128 * D * 2, QTILE = 64 * D * 2;
  static constexpr int NS = D == 128 ? 4 : 8;  // stages of Q and dO tiles
  static constexpr int OFF_K = 0, OFF_V = KTILE, OFF_RING = 2 * KTILE;
  static constexpr int OFF_STAT = OFF_RING + NS * 2 * QTILE;  // float2 [NS][64]: base-2 lse, delta
  static constexpr int OFF_BAR = OFF_STAT + NS * 512;
  static constexpr int B_FULL = 0, B_EMPTY = B_FULL + NS, B_STAT = B_EMPTY + NS, B_KV = B_STAT + NS;
  static constexpr int B_SD = B_KV + 1;  // [2] S^T and dP^T ready (commit)
  static constexpr int B_PD = B_SD + 2;  // [2] P^T and dS^T written (4 warps)
  static constexpr int B_O = B_PD + 2;
  static constexpr int NBARS = B_O + 1;
  static constexpr int OFF_MISC = OFF_BAR + 8 * NBARS;  // tmem, abort, kt, run, runs, slot
  static constexpr int SMEM = OFF_MISC + 32 + 1024;
  static constexpr int DV_COL = 0, DK_COL = 128, S_COL = 256, DP_COL = 384;  // two 64-column buffers each
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

template <int D>
__global__ void __launch_bounds__(384, 1)
attend_dkv_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmG,
                  const AttendGradParams p) {
  using C = AttendDkvCfg<D>;
  using namespace tc;
  extern __shared__ __align__(16) uint8_t attend_dkv_smem[];
  const uint32_t raw_u = smem_u32(attend_dkv_smem);
  const uint32_t base_u = (raw_u + 1023u) & ~1023u;
  uint8_t* base = attend_dkv_smem + (base_u - raw_u);
  int* misc = reinterpret_cast<int*>(base + C::OFF_MISC);
  volatile int* abort_flag = misc + 1;
  const uint32_t bar0 = base_u + C::OFF_BAR;
  asm volatile("griddepcontrol.launch_dependents;");
#define ABAR(i) (bar0 + 8u * uint32_t(i))
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.Hq / p.Hkv, BH = p.B * p.Hkv;
  const int bh = blockIdx.x % BH;  // the heads' heaviest runs (first tokens, causal) go first
  const int b = bh / p.Hkv, hk = bh % p.Hkv;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(ABAR(C::B_FULL + s), 1);
      mbar_init(ABAR(C::B_EMPTY + s), 1);
      mbar_init(ABAR(C::B_STAT + s), 1);
    }
    mbar_init(ABAR(C::B_KV), 1);
    for (int g = 0; g < 2; ++g) {
      mbar_init(ABAR(C::B_SD + g), 1);
      mbar_init(ABAR(C::B_PD + g), 4);
    }
    mbar_init(ABAR(C::B_O), 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 2) {
    tmem_alloc(base_u + C::OFF_MISC, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  if (warp == 3) {
    const RunAt f = find_run(p, blockIdx.x / BH, -1);
    if (lane == 0) {
      misc[2] = f.kt;
      misc[3] = f.run;
      misc[4] = f.runs;
      misc[5] = f.slot;
    }
  }
  // the setup ran beside the dQ kernel's last blocks; delta is that kernel's
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uint32_t(misc[0]);
  const int kt = misc[2], run = misc[3], runs = misc[4];
  const QueryRange range(p.win, kt, p.N);
  const long long total = (long long)(G)*range.count;
  const int from = int(total * run / runs), to = int(total * (run + 1) / runs);
  const int j0 = kt * 128;

  if (warp == 0) {
    // lanes 0 and 1: the two 64-column panels
    if (lane < 2) {
      bool ok = true;
      if (lane == 0) mbar_arrive_expect_tx(ABAR(C::B_KV), 2 * C::KTILE);
      __syncwarp(0x3u);
      if (lane * 64 < D) {
        tma_load_3d(base_u + C::OFF_K + lane * 16384, &tmK, ABAR(C::B_KV), lane * 64, j0, bh);
        tma_load_3d(base_u + C::OFF_V + lane * 16384, &tmV, ABAR(C::B_KV), lane * 64, j0, bh);
      }
      int use = 0;
      for (int i = from; i < to; ++i, ++use) {
        const int s = use % C::NS;
        ok = wait_bounded(ABAR(C::B_EMPTY + s), ((use / C::NS) & 1) ^ 1, abort_flag);
        ok = __all_sync(0x3u, ok);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(ABAR(C::B_FULL + s), 2 * C::QTILE);
        __syncwarp(0x3u);
        const int head = b * p.Hq + hk * G + i / range.count, q0 = (range.first + i % range.count) * 64;
        const uint32_t dst = base_u + C::OFF_RING + s * 2 * C::QTILE;
        if (lane * 64 < D) {
          tma_load_3d(dst + lane * 8192, &tmQ, ABAR(C::B_FULL + s), lane * 64, q0, head);
          tma_load_3d(dst + C::QTILE + lane * 8192, &tmG, ABAR(C::B_FULL + s), lane * 64, q0, head);
        }
      }
      if (lane == 0) {
        wait_drain(ABAR(C::B_KV), 0);
        for (int u = use > C::NS ? use - C::NS : 0; u < use; ++u) wait_drain(ABAR(C::B_FULL + u % C::NS), (u / C::NS) & 1);
      }
    }
  } else if (warp == 1) {
    constexpr uint32_t idS = idesc_bf16(128, 64, false), idG = idesc_bf16(128, D, true);
    const bool lead = elect();
    const int count = to - from;
    auto stage = [&](int i) { return base_u + C::OFF_RING + (i % C::NS) * 2 * C::QTILE; };
    auto scores = [&](int i) -> bool {  // S^T = K Q^T, dP^T = V dO^T of the run's i-th tile
      if (!wait_warp(ABAR(C::B_FULL + i % C::NS), (i / C::NS) & 1, abort_flag)) return false;
      tc_fence_after();
      if (lead) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint64_t a = operand(base_u + (w ? C::OFF_V : C::OFF_K), 16), q = operand(stage(i) + w * C::QTILE, 16);
#pragma unroll
          for (int c = 0; c < D / 16; ++c)
            umma_ss(tmem + (w ? C::DP_COL : C::S_COL) + (i & 1) * 64, a + (((c >> 2) * 16384 + (c & 3) * 32) >> 4),
                    q + (((c >> 2) * 8192 + (c & 3) * 32) >> 4), idS, c ? 1u : 0u);
        }
        umma_commit(ABAR(C::B_SD + (i & 1)));
      }
      return true;
    };
    bool ok = wait_warp(ABAR(C::B_KV), 0, abort_flag);
    if (ok) ok = scores(0);
    if (ok && count > 1) ok = scores(1);
    for (int i = 0; i < count && ok; ++i) {
      if (!(ok = wait_warp(ABAR(C::B_PD + (i & 1)), (i >> 1) & 1, abort_flag))) break;
      tc_fence_after();
      if (lead) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint64_t q = operand(stage(i) + (w ? 0 : C::QTILE), 8192);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            umma_ts(tmem + (w ? C::DK_COL : C::DV_COL), tmem + (w ? C::DP_COL : C::S_COL) + (i & 1) * 64 + c * 8,
                    q + c * (2048 >> 4), idG, (i | c) ? 1u : 0u);
        }
        umma_commit(ABAR(C::B_EMPTY + i % C::NS));
      }
      if (i + 2 < count) ok = scores(i + 2);
    }
    if (lead) {
      umma_commit(ABAR(C::B_O));
      wait_drain(ABAR(C::B_O), 0);
    }
    __syncwarp();
  } else if (warp == 2) {
    // each tile's row statistics; rows behind the last one weigh nothing
    for (int i = from, use = 0; i < to; ++i, ++use) {
      const int s = use % C::NS;
      const int head = b * p.Hq + hk * G + i / range.count, q0 = (range.first + i % range.count) * 64;
      float2 x[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int t = q0 + k * 32 + lane;
        const size_t row = size_t(head) * p.N + t;
        x[k] = t < p.N ? make_float2(p.lse[row] * 1.4426950408889634f, p.delta[row]) : make_float2(INFINITY, 0.f);
      }
      if (!__all_sync(0xffffffffu, wait_bounded(ABAR(C::B_EMPTY + s), ((use / C::NS) & 1) ^ 1, abort_flag))) break;
      float2* st = reinterpret_cast<float2*>(base + C::OFF_STAT) + s * 64;
      st[lane] = x[0];
      st[32 + lane] = x[1];
      warp_arrive(ABAR(C::B_STAT + s));
    }
  } else if (warp >= 4) {
    const int g = (warp - 4) >> 2, j = j0 + (threadIdx.x & 127);
    const uint32_t lrow = uint32_t((warp & 3) * 32) << 16;
    const float sl2 = p.scale * 1.4426950408889634f;
    const int count = to - from;
    // the rows that see key j: positions [lo, hi]
    const int lo = max(0, j - p.win.right);
    const int hi = j < p.win.sinks ? p.N - 1 : int(min((long long)p.N - 1, (long long)j + p.win.left));
    bool ok = true;
    for (int i = g; i < count; i += 2) {
      const int q0 = (range.first + (from + i) % range.count) * 64, s = i % C::NS;
      const bool whole = q0 >= j0 + 127 - p.win.right && q0 + 63 < p.N && j0 + 127 < p.N &&
                         (j0 + 128 <= p.win.sinks || q0 + 63 <= (long long)j0 + p.win.left);
      ok = __all_sync(0xffffffffu, wait_bounded(ABAR(C::B_STAT + s), (i / C::NS) & 1, abort_flag) &&
                                       wait_bounded(ABAR(C::B_SD + g), (i >> 1) & 1, abort_flag));
      if (!ok) break;
      tc_fence_after();
      const uint32_t sa = tmem + lrow + C::S_COL + g * 64, da = tmem + lrow + C::DP_COL + g * 64;
      uint32_t sc[64], dp[64];
#pragma unroll
      for (int ch = 0; ch < 4; ++ch) {
        tmem_ld16(sa + ch * 16, *reinterpret_cast<uint32_t(*)[16]>(&sc[ch * 16]));
        tmem_ld16(da + ch * 16, *reinterpret_cast<uint32_t(*)[16]>(&dp[ch * 16]));
      }
#pragma unroll
      for (int ch = 0; ch < 4; ++ch) {
        tmem_wait_ld(*reinterpret_cast<uint32_t(*)[16]>(&sc[ch * 16]));
        tmem_wait_ld(*reinterpret_cast<uint32_t(*)[16]>(&dp[ch * 16]));
      }
      const float4* st = reinterpret_cast<const float4*>(base + C::OFF_STAT + s * 512);
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const float4 x = st[k];  // base-2 lse and delta of two rows
        const float w0 = ex2(fmaf(__uint_as_float(sc[2 * k]), sl2, -x.x));
        const float w1 = ex2(fmaf(__uint_as_float(sc[2 * k + 1]), sl2, -x.z));
        dp[2 * k] = __float_as_uint(w0 * (__uint_as_float(dp[2 * k]) - x.y));
        dp[2 * k + 1] = __float_as_uint(w1 * (__uint_as_float(dp[2 * k + 1]) - x.w));
        sc[2 * k] = __float_as_uint(w0);
        sc[2 * k + 1] = __float_as_uint(w1);
      }
      if (!whole) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint32_t bits = ones_below(hi - q0 + 1 - 32 * w) & ~ones_below(lo - q0 - 32 * w);
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (!((bits >> k) & 1u)) sc[32 * w + k] = dp[32 * w + k] = 0u;
        }
      }
#pragma unroll
      for (int ch = 0; ch < 2; ++ch) {
        uint32_t pk[16];
#pragma unroll
        for (int k = 0; k < 16; ++k)
          pk[k] = pack_bf16x2(__uint_as_float(sc[ch * 32 + 2 * k]), __uint_as_float(sc[ch * 32 + 2 * k + 1]));
        tmem_st16(sa + ch * 16, pk);
#pragma unroll
        for (int k = 0; k < 16; ++k)
          pk[k] = pack_bf16x2(__uint_as_float(dp[ch * 32 + 2 * k]), __uint_as_float(dp[ch * 32 + 2 * k + 1]));
        tmem_st16(da + ch * 16, pk);
      }
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(ABAR(C::B_PD + g));
    }
    ok = __all_sync(0xffffffffu, ok && wait_bounded(ABAR(C::B_O), 0, abort_flag));
    tc_fence_after();
    // group 0 writes dV, group 1 dK
    const float f = g ? p.scale : 1.f;
    const uint32_t col = tmem + lrow + (g ? C::DK_COL : C::DV_COL);
    const size_t key = size_t(bh) * p.N + j;
    float* part = p.part + (size_t(bh) * p.slots + misc[5] + run) * (2 * 128 * D) + g * 128 * D;
    bf16* out = g ? p.dK : p.dV;
#pragma unroll 1
    for (int ch = 0; ch < D / 32; ++ch) {
      __syncwarp();
      uint32_t x[2][16];
      tmem_ld16(col + ch * 32, x[0]);
      tmem_ld16(col + ch * 32 + 16, x[1]);
      tmem_wait_ld(x[0]);
      tmem_wait_ld(x[1]);
      if (runs > 1) store_part32(part + ch * 32, ok ? int64_t(threadIdx.x & 127) * D : -1, x, f);
      else store_rows32(out + ch * 32, ok && j < p.N ? int64_t(key) * D : -1, x, f);
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
#undef ABAR
}

// Adds up the runs of the key tiles that were cut, in run order: kJoinSlices blocks per key tile and
// key head, each a slice of its dV and dK, a row's 4 columns per thread and step.
constexpr int kJoinSlices = 16;
template <int D>
__global__ void __launch_bounds__(256) attend_dkv_join_kernel(const AttendGradParams p) {
  const int kts = (p.N + 127) / 128, kt = blockIdx.x / kJoinSlices % kts, bh = blockIdx.x / kJoinSlices / kts;
  const bool cut = query_runs((p.Hq / p.Hkv) * QueryRange(p.win, kt, p.N).count, p.run) > 1;
  RunAt f{};
  if (cut) f = find_run(p, -1, kt);  // every warp finds the same
  // every block waits, so that this grid does not end before the one it depends on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!cut) return;
  constexpr int ALL = 2 * 128 * D, SLICE = ALL / kJoinSlices;
  const float* src = p.part + (size_t(bh) * p.slots + f.slot) * ALL;
  for (int e = blockIdx.x % kJoinSlices * SLICE + threadIdx.x * 4, end = (blockIdx.x % kJoinSlices + 1) * SLICE; e < end; e += 1024) {
    const int g = e / (128 * D), j = kt * 128 + (e / D) % 128, c = e % D;
    if (j >= p.N) continue;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int r = 0; r < f.runs; ++r) {
      const float4 x = *reinterpret_cast<const float4*>(src + size_t(r) * ALL + e);
      a.x += x.x;
      a.y += x.y;
      a.z += x.z;
      a.w += x.w;
    }
    *reinterpret_cast<uint2*>((g ? p.dK : p.dV) + (size_t(bh) * p.N + j) * D + c) =
        make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
  }
}

}  // namespace pisa
