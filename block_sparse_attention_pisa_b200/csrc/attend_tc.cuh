// Attention under a token-exact window on the tensor cores (tcgen05 / TMEM / TMA), over keys
// laid out plainly or in pages.
//
//   o = sum_j exp(s_j - m) v_j / l,  l = sum_j exp(s_j - m),  s_j = scale q.k_j, j visible
//
// one pass over the keys with a running maximum m and sum l per row.
//
// A persistent CTA per SM takes items in turn: a tile of 128 rows of one key head that walks the
// 128-key tiles that some row of it sees (the tiles of the first tokens, then the window's), or
// one run of them. Warp roles:
//   warp 0       producer: K and V tiles by TMA (a page at a time in a paged cache) into a ring,
//                running ahead into the next items;
//   warp 1       issues every tcgen05.mma: per tile S = Q K^T, then O += P V, both with the first
//                operand in tensor memory;
//   warp 2       paged caches: clears the rows of a V tile that no row may see (unwritten rows
//                may hold anything, and 0 x NaN is NaN); 8 bits: warps 2-3 turn codes into
//                operands;
//   warps 4-11   softmax: two threads per row (warps w and w + 4), each with 64 keys of a tile
//                and half of O's columns; they load the queries and write the output.
// Tensor memory: O (D columns), the queries (D/2, 16-bit pairs), two buffers of S (128 columns
// each); P in 16 bits overwrites the start of each half of its own S.
//
// S of tile i + 1 goes to the other buffer and is issued before P of tile i is awaited, so the
// scores of the next tile are there when a softmax ends, and the products run under the
// exponentials. The next item's queries are put into tensor memory as soon as the last scores of
// this one are in, so its first scores run under this item's last softmax and output too. Products
// are issued by one lane and execute in order: S of tile i + 2 may overwrite P of tile i behind
// the P V that reads it. The two threads of a row agree by a vote per tile; only when one of them
// sees the maximum grow by more than 2^8 do they exchange maxima and rescale O.
//
// Bound at D = 128: a tile of 128 x 128 takes 2 x 512 cycles of tensor time and 1024 on the
// exponential unit (16 per cycle and SM); shared memory carries 128 KB for it (K and V written
// and read once), 1024 cycles at 128 bytes. With the queries in shared memory it would be 160 KB.
// Before, two tiles of 128 rows alternated with one buffer of S each: the chain softmax -> P V
// -> next scores took 4100 cycles for the two (window_image in the measured cases: 157 us).
#pragma once

#include "attention_tc.cuh"
#include "window.cuh"

namespace pisa {

// A tile of 128 rows holds `tokens` consecutive tokens of all query heads of a key head (of up to
// 128 of them), head by head: row r is head r / tokens, token r % tokens. Shared keys are read once
// for all their heads, and a tile spans few positions; with a group that does not divide 128 a
// few rows stay idle (3 heads: 2).
struct RowTiles {
  int tokens, heads, parts;  // heads of a tile; tiles that a group's heads take
  __host__ __device__ static RowTiles of(int G) {
    const int h = G < 128 ? G : 128;
    return RowTiles{128 / h, h, (G + 127) / 128};
  }
};

struct AttendTcParams {
  const bf16* Q;
  bf16* O;
  float* lse;
  float* part;      // splits > 1: fp32 [splits][B * Hq * N][D], then base-2 lse [splits][B * Hq * N]
  float* part_lse;
  Pages pages;      // paged only
  int B, Hq, Hkv, N;
  RowTiles rt;
  int tiles;        // row tiles of a key head
  int splits;       // runs that a row tile's key tiles are cut into
  int items;        // tiles * B * Hkv * splits
  Window win;
  float scale;
};

template <int D, int KV>
struct AttendTcCfg {
  static constexpr bool CODES = KV == kKvPagedE4m3;
  static constexpr int kThreads = 384;
  static constexpr int TILE = 128 * D * 2;          // bytes of a 128-row 16-bit tile
  static constexpr int NS = (CODES ? 4 : 6) * (128 / D);  // ring stages
  static constexpr int NL = CODES ? 4 * (128 / D) : NS;   // landing stages (8 bits: tiles of codes)
  static constexpr int LAND = CODES ? 128 * D : 0;  // bytes of a landing stage of its own
  static constexpr int CONVERTERS = 2;              // warps
  static constexpr int OFF_RING = 0;
  static constexpr int OFF_CODES = OFF_RING + NS * TILE;
  static constexpr int OFF_SCALE = OFF_CODES + NL * LAND;  // 8 bits: float [8 warps][K, V][64]
  static constexpr int OFF_X = OFF_SCALE + (CODES ? 8 * 2 * 64 * 4 : 0);  // float [2][128]: a pair's exchange
  static constexpr int OFF_BAR = OFF_X + 1024;
  static constexpr int B_FULL = 0;                  // [NS] stage holds its tile
  static constexpr int B_EMPTY = B_FULL + NS;       // [NS] products that read it are done (commit)
  static constexpr int B_LAND = B_EMPTY + NS;       // [NL] paged: copies landed, rows not cleared yet
  static constexpr int B_LEMPTY = B_LAND + NL;      // [NL] 8 bits: codes converted
  static constexpr int B_Q = B_LEMPTY + NL;         // queries are in tensor memory (8 warps)
  static constexpr int B_S = B_Q + 1;               // [2] S ready (commit)
  static constexpr int B_P = B_S + 2;               // [2] P written (8 warps)
  static constexpr int B_O = B_P + 2;               // the item's last product is done (commit)
  static constexpr int B_END = B_O + 1;             // all products done (commit)
  static constexpr int NBARS = B_END + 1;
  static constexpr int OFF_MISC = OFF_BAR + 8 * NBARS;
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
  static constexpr int O_COL = 0, Q_COL = 128, S_COL = 192;
  static_assert(SMEM <= 227 * 1024, "shared memory budget");
};

// What a group of rows sees: sinks [0, sk) and window [lo, hi); rows at positions p0 .. p1.
struct Sight {
  int p0, p1, lo, hi, sk;
  __device__ __forceinline__ void set(const Window& w, int first, int last, int n) {
    p0 = first;
    p1 = last;
    hi = max(0, min(n, last + w.right + 1));
    lo = min(hi, max(0, first - w.left));
    sk = min(w.sinks, hi);
  }
  __device__ __forceinline__ void none() { p0 = p1 = lo = hi = sk = 0; }
  // some row may see a key of [j0, j0 + 128)
  __device__ __forceinline__ bool any(int j0) const { return j0 < sk || (j0 < hi && j0 + 128 > lo); }
  // some row may see a key of [j0, j0 + w)
  __device__ __forceinline__ bool any(int j0, int w) const { return j0 < sk || (j0 < hi && j0 + w > lo); }
};

// The tiles of 128 keys that two groups see together, split into runs.
struct TileList {
  int ns, first, from, to;  // sink tiles before the window's, window's first tile, this run
  __device__ __forceinline__ void set(const Sight& a, int split, int splits) {
    const int w0 = a.lo >> 7, w1 = a.hi > a.lo ? (a.hi + 127) >> 7 : w0;
    ns = min((a.sk + 127) >> 7, w0);
    first = w0;
    const long long total = ns + (w1 - w0);
    from = int(total * split / splits);
    to = int(total * (split + 1) / splits);
  }
  __device__ __forceinline__ int key(int i) const { return (i < ns ? i : first + i - ns) << 7; }
};

__device__ __forceinline__ uint32_t ones_below(int k) {  // bits [0, k) of a word, any k
  return k <= 0 ? 0u : (k >= 32 ? 0xffffffffu : (1u << k) - 1u);
}

// pages of the tile at j0 that `a` may see and the table holds: bit i = page i of the tile
__device__ __forceinline__ uint32_t held_pages(const Pages& g, int b, const Sight& a, int j0, int lane) {
  const int per = 128 >> g.log_page;
  bool ok = false;
  if (lane < per) {
    const int j = j0 + (lane << g.log_page);
    ok = a.any(j, 1 << g.log_page) && page_of(g, b, j) >= 0;
  }
  return __ballot_sync(0xffffffffu, ok);
}

// A 128-byte swizzled operand at `saddr` as its descriptor; a product's step adds its offset in
// 16-byte units to the low word. All lanes of the issuing warp run the loop and hold the same
// values, so that they stay in uniform registers; one lane issues. (With the loop in one lane's
// branch each product took about 95 cycles to issue against 64 to execute.)
__device__ __forceinline__ uint64_t operand(uint32_t saddr, uint32_t lbo) { return tc::sdesc_sw128(saddr, lbo, 1024); }
__device__ __forceinline__ bool elect() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}
// wait of a whole warp that issues products
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, tc::wait_poll(bar, parity, abort_flag));
}

// 4 x 4 transposition of 16-byte pieces among the lanes of a quad
__device__ __forceinline__ void transpose_quads(uint32_t (&c)[4][4]) {
#pragma unroll
  for (int d = 1; d <= 2; ++d)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int a = d == 1 ? 2 * e : e, b = a + d;
      const bool high = (threadIdx.x & d) != 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? c[a][k] : c[b][k], d);
        if (high) c[a][k] = got;
        else c[b][k] = got;
      }
    }
}

// 32 fp32 columns of a warp's 32 rows (lane = row) as bf16 at dst[row] + 0 .. 31. The lanes of a
// quad exchange 16-byte pieces so that each store covers 64 contiguous bytes of eight rows, not 16
// of 32 (5000 cycles for a tile of 128 x 128 at one row per lane). `at`: element offset of this
// lane's row, < 0 if it is not written.
__device__ __forceinline__ void store_rows32(bf16* dst, int64_t at, const uint32_t (&x)[2][16], float scale) {
  uint32_t c[4][4];
#pragma unroll
  for (int k = 0; k < 16; ++k)
    c[k >> 2][k & 3] = pack_bf16x2(__uint_as_float(x[k >> 3][(2 * k) & 15]) * scale, __uint_as_float(x[k >> 3][(2 * k + 1) & 15]) * scale);
  const int q = threadIdx.x & 3;
  transpose_quads(c);
#pragma unroll
  for (int j = 0; j < 4; ++j) {  // piece q of the quad's row j
    const int64_t to = __shfl_sync(0xffffffffu, at, (threadIdx.x & 28) + j);
    if (to >= 0) *reinterpret_cast<uint4*>(dst + to + q * 8) = make_uint4(c[j][0], c[j][1], c[j][2], c[j][3]);
  }
}

// fp32 pairs: x = x * a + b, sum += x
__device__ __forceinline__ void fma2(float& x0, float& x1, float a, float b) {
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmov.b64 z, {%3, %3};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(a), "f"(b));
}
__device__ __forceinline__ void add2(float& s0, float& s1, float x0, float x1) {
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(s0), "+f"(s1)
      : "f"(x0), "f"(x1));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 32 fp32 columns of a warp's 32 rows (lane = row) to dst[at] + 0 .. 31, in pieces as store_rows32
__device__ __forceinline__ void store_part32(float* dst, int64_t at, const uint32_t (&x)[2][16], float scale) {
  const int q = threadIdx.x & 3;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t c[4][4];
#pragma unroll
    for (int k = 0; k < 16; ++k) c[k >> 2][k & 3] = __float_as_uint(__uint_as_float(x[h][k]) * scale);
    transpose_quads(c);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t to = __shfl_sync(0xffffffffu, at, (threadIdx.x & 28) + j);
      if (to >= 0) *reinterpret_cast<uint4*>(dst + to + h * 16 + q * 4) = make_uint4(c[j][0], c[j][1], c[j][2], c[j][3]);
    }
  }
}

// fp16 operands: idesc_bf16 with the 16-bit format of both operands fp16
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N) { return tc::idesc_bf16(M, N, false) & ~((1u << 7) | (1u << 10)); }

// One piece of work: a row tile of a key head over one run of its key tiles.
struct AttendItem {
  int b, hk, bh, split, n, nq;
  int t0, head0, heads;  // first token; first query head and how many are real
  Sight see;
  TileList tiles;
  bool real;             // has a row
  __device__ __forceinline__ bool live() const { return real && tiles.to > tiles.from; }
};
template <int KV>
__device__ __forceinline__ AttendItem attend_item(const AttendTcParams& p, int id) {
  AttendItem w;
  const int G = p.Hq / p.Hkv;
  int tile = id % p.tiles;
  id /= p.tiles;
  w.split = id % p.splits;
  w.bh = id / p.splits;
  w.b = w.bh / p.Hkv;
  w.hk = w.bh - w.b * p.Hkv;
  w.n = w.nq = p.N;
  if constexpr (KV != kKvPlain) {
    w.n = kv_len_of(p.pages, w.b);
    w.nq = q_len_of(p.pages, w.b, p.N);
  }
  int part = 0;
  const int per = p.tiles / p.rt.parts;
  if (p.rt.parts > 1) {
    part = tile / per;
    tile -= part * per;
  }
  w.t0 = (per - 1 - tile) * p.rt.tokens;  // causal: the rows with the most keys first
  w.head0 = w.b * p.Hq + w.hk * G + part * 128;
  w.heads = min(p.rt.heads, G - part * 128);
  w.real = w.t0 < w.nq;
  if (w.real) w.see.set(p.win, w.n - w.nq + w.t0, w.n - w.nq + min(w.t0 + p.rt.tokens, w.nq) - 1, w.n);
  else w.see.none();
  w.tiles.set(w.see, w.split, p.splits);
  return w;
}
// the first live item from `id` on (id moves to it, past the end if there is none)
template <int KV>
__device__ __forceinline__ AttendItem live_item(const AttendTcParams& p, int& id) {
  AttendItem w = attend_item<KV>(p, min(id, p.items - 1));
  while (id < p.items && !w.live()) {
    id += int(gridDim.x);
    w = attend_item<KV>(p, min(id, p.items - 1));
  }
  return w;
}

template <int D, int KV>
__global__ void __launch_bounds__(384, 1)
attend_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                 const AttendTcParams p) {
  using C = AttendTcCfg<D, KV>;
  using namespace tc;
  extern __shared__ __align__(16) uint8_t attend_smem[];
  const uint32_t raw_u = smem_u32(attend_smem);
  const uint32_t base_u = (raw_u + 1023u) & ~1023u;
  uint8_t* base = attend_smem + (base_u - raw_u);
  volatile int* abort_flag = reinterpret_cast<int*>(base + C::OFF_MISC) + 1;
  const uint32_t bar0 = base_u + C::OFF_BAR;
#define ABAR(i) (bar0 + 8u * uint32_t(i))
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int items = p.items, step = int(gridDim.x);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::NS; ++s) {
      mbar_init(ABAR(C::B_FULL + s), C::CODES ? C::CONVERTERS : 1);
      mbar_init(ABAR(C::B_EMPTY + s), 1);
    }
    for (int s = 0; s < C::NL; ++s) {
      mbar_init(ABAR(C::B_LAND + s), 1);
      mbar_init(ABAR(C::B_LEMPTY + s), C::CONVERTERS);
    }
    mbar_init(ABAR(C::B_Q), 8);
    for (int g = 0; g < 2; ++g) {
      mbar_init(ABAR(C::B_S + g), 1);
      mbar_init(ABAR(C::B_P + g), 8);
    }
    mbar_init(ABAR(C::B_O), 1);
    mbar_init(ABAR(C::B_END), 1);
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

  // Every role walks the CTA's items; the n-th key tile of them all has K as stage use 2 n and V as
  // 2 n + 1, and S buffer n % 2.
  if (warp == 0) {
    // ------------------------------------------------------------- producer
    // lanes 0 and 1 issue the two 64-column panels of a tile (D = 64: lane 0 alone)
    if (lane < 2) {
      bool ok = true;
      int use = 0;
      constexpr int NL = C::NL;  // the stages that the copies land in: the ring's, or those for codes
      for (int id = blockIdx.x; id < items && ok; id += step) {
        const AttendItem w = attend_item<KV>(p, id);
        for (int i = w.tiles.from; i < w.tiles.to && ok; ++i) {
          const int j0 = w.tiles.key(i);
          for (int kv = 0; kv < 2 && ok; ++kv, ++use) {
            const int s = use % NL;
            ok = wait_bounded(ABAR((C::CODES ? C::B_LEMPTY : C::B_EMPTY) + s), ((use / NL) & 1) ^ 1, abort_flag);
            ok = __all_sync(0x3u, ok);
            if (!ok) break;
            const uint32_t dst = base_u + (C::CODES ? C::OFF_CODES + s * C::LAND : C::OFF_RING + s * C::TILE);
            if constexpr (KV == kKvPlain) {
              if (lane == 0) mbar_arrive_expect_tx(ABAR(C::B_FULL + s), C::TILE);
              __syncwarp(0x3u);
              if (lane * 64 < D)
                tma_load_3d(dst + lane * 16384, kv ? &tmV : &tmK, ABAR(C::B_FULL + s), lane * 64, j0, w.bh);
            } else {
              // pages that no row of the tile sees, or that the table does not hold, stay out
              const int per = 128 >> p.pages.log_page, size = 1 << p.pages.log_page;
              uint32_t held = 0;
              for (int q = 0; q < per; ++q)
                if (w.see.any(j0 + q * size, size) && page_of(p.pages, w.b, j0 + q * size) >= 0) held |= 1u << q;
              if (lane == 0) mbar_arrive_expect_tx(ABAR(C::B_LAND + s), __popc(held) * size * D * (C::CODES ? 1 : 2));
              __syncwarp(0x3u);
              if constexpr (C::CODES) {  // whole rows of D codes, lanes by turns
                for (int q = lane; q < per; q += 2)
                  if ((held >> q) & 1u)
                    tma_load_3d(dst + q * size * D, kv ? &tmV : &tmK, ABAR(C::B_LAND + s), 0, 0,
                                page_of(p.pages, w.b, j0 + q * size) * p.Hkv + w.hk);
              } else if (lane * 64 < D) {
                for (int q = 0; q < per; ++q)
                  if ((held >> q) & 1u)
                    tma_load_3d(dst + lane * 16384 + q * size * 128, kv ? &tmV : &tmK, ABAR(C::B_LAND + s), lane * 64, 0,
                                page_of(p.pages, w.b, j0 + q * size) * p.Hkv + w.hk);
              }
            }
          }
        }
      }
      // no copy may still be in flight when the CTA exits
      constexpr int landed = KV == kKvPlain ? C::B_FULL : C::B_LAND;
      if (lane == 0)
        for (int u = use > NL ? use - NL : 0; u < use; ++u) wait_drain(ABAR(landed + u % NL), (u / NL) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------- products
    constexpr uint32_t idS = C::CODES ? idesc_f16(128, 128) : idesc_bf16(128, 128, false), idO = idesc_bf16(128, D, true);
    const bool lead = elect();
    auto full = [&](int u) { return wait_warp(ABAR(C::B_FULL + u % C::NS), (u / C::NS) & 1, abort_flag); };
    int id = blockIdx.x, next_id = id;
    AttendItem w = live_item<KV>(p, id), next = w;
    bool ok = true, prev = false, prev_first = false, prev_last = false;
    int i = 0;           // the item's tile whose scores come next
    uint32_t n_q = 0;    // phase of the queries
    for (int n = 0; ok; ++n) {
      const bool more = id < items;
      const bool first = i == 0, last = i == w.tiles.to - w.tiles.from - 1;
      if (more) {  // S = Q K^T of tile n
        if (first) {
          if (!(ok = wait_warp(ABAR(C::B_Q), n_q, abort_flag))) break;
          n_q ^= 1u;
        }
        if (!(ok = full(2 * n))) break;
        tc_fence_after();
        if (lead) {
          const uint64_t k = operand(base_u + C::OFF_RING + ((2 * n) % C::NS) * C::TILE, 16);
#pragma unroll
          for (int c = 0; c < D / 16; ++c)
            umma_ts(tmem + C::S_COL + (n & 1) * 128, tmem + C::Q_COL + c * 8, k + (((c >> 2) * 16384 + (c & 3) * 32) >> 4), idS,
                    c ? 1u : 0u);
          umma_commit(ABAR(C::B_S + (n & 1)));
          umma_commit(ABAR(C::B_EMPTY + (2 * n) % C::NS));
        }
        if (first) {  // while the products run
          next_id = id + step;
          next = live_item<KV>(p, next_id);
        }
      }
      if (prev) {  // O += P V of tile n - 1
        if (!(ok = full(2 * n - 1))) break;
        if (!(ok = wait_warp(ABAR(C::B_P + ((n - 1) & 1)), ((n - 1) >> 1) & 1, abort_flag))) break;
        tc_fence_after();
        if (lead) {
          const uint64_t v = operand(base_u + C::OFF_RING + ((2 * n - 1) % C::NS) * C::TILE, 16384);
          const uint32_t pa = tmem + C::S_COL + ((n - 1) & 1) * 128;
          // keys [16c, 16c + 16): the thread of half c / 4 packed them at the start of its columns
#pragma unroll
          for (int c = 0; c < 8; ++c)
            umma_ts(tmem + C::O_COL, pa + (c >> 2) * 64 + (c & 3) * 8, v + c * (2048 >> 4), idO, (c || !prev_first) ? 1u : 0u);
          umma_commit(ABAR(C::B_EMPTY + (2 * n - 1) % C::NS));
          if (prev_last) umma_commit(ABAR(C::B_O));
        }
      }
      if (!more) break;
      prev = true;
      prev_first = first;
      prev_last = last;
      ++i;
      if (last) {
        w = next;
        id = next_id;
        i = 0;
      }
    }
    if (lead) {
      umma_commit(ABAR(C::B_END));
      wait_drain(ABAR(C::B_END), 0);  // nothing of ours may run on after the CTA frees TMEM
    }
    __syncwarp();
  } else if (warp < 4) {
    // ------------------------------------------------------------- paged: rows nobody may see, codes
    bool ok = true;
    int use = 0;
    if constexpr (KV == kKvPagedE4m3) {
      // 16 codes per thread and step -> 32 bytes of the swizzled operand (keys in fp16, values in
      // bf16: their weights need its range); rows that nobody may see become zero. The scales stay
      // out: scores and weights take them exactly in fp32.
      const int ct = threadIdx.x - 64;
      constexpr int CH = D / 16, NT = 32 * C::CONVERTERS;  // 16-code chunks of a row
      for (int id = blockIdx.x; id < items && ok; id += step) {
        const AttendItem w = attend_item<KV>(p, id);
        for (int i = w.tiles.from; i < w.tiles.to && ok; ++i) {
          const int j0 = w.tiles.key(i);
          const uint32_t held = held_pages(p.pages, w.b, w.see, j0, lane);
          const bool inner = (j0 + 128 <= w.see.sk || (j0 >= w.see.lo && j0 + 128 <= w.see.hi)) &&
                             held == (1u << (128 >> p.pages.log_page)) - 1u;
          for (int kv = 0; kv < 2; ++kv, ++use) {
            const int sl = use % C::NL, s = use % C::NS;
            ok = wait_bounded(ABAR(C::B_EMPTY + s), ((use / C::NS) & 1) ^ 1, abort_flag) &&
                 wait_bounded(ABAR(C::B_LAND + sl), (use / C::NL) & 1, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
#pragma unroll 4
            for (int x = ct; x < 128 * CH; x += NT) {
              const int r = x / CH, c = x % CH, j = j0 + r;
              uint4 code = *reinterpret_cast<const uint4*>(base + C::OFF_CODES + sl * C::LAND + r * D + c * 16);
              if (!inner) {
                const bool in = ((held >> (r >> p.pages.log_page)) & 1u) && (j < w.see.sk || (j >= w.see.lo && j < w.see.hi));
                if (!in) code = make_uint4(0, 0, 0, 0);
              }
              uint4 lo, hi;
              if (kv) {
                lo = make_uint4(e4m3x2_to_bf16x2(code.x), e4m3x2_to_bf16x2(code.x >> 16), e4m3x2_to_bf16x2(code.y),
                                e4m3x2_to_bf16x2(code.y >> 16));
                hi = make_uint4(e4m3x2_to_bf16x2(code.z), e4m3x2_to_bf16x2(code.z >> 16), e4m3x2_to_bf16x2(code.w),
                                e4m3x2_to_bf16x2(code.w >> 16));
              } else {
                lo = make_uint4(codes_to_f16_lo(code.x), codes_to_f16_hi(code.x), codes_to_f16_lo(code.y), codes_to_f16_hi(code.y));
                hi = make_uint4(codes_to_f16_lo(code.z), codes_to_f16_hi(code.z), codes_to_f16_lo(code.w), codes_to_f16_hi(code.w));
              }
              uint8_t* dst = base + C::OFF_RING + s * C::TILE + (c >> 2) * 16384 + r * 128;
              const int c0 = (2 * c) & 7;
              *reinterpret_cast<uint4*>(dst + ((c0 ^ (r & 7)) << 4)) = lo;
              *reinterpret_cast<uint4*>(dst + (((c0 + 1) ^ (r & 7)) << 4)) = hi;
            }
            fence_proxy_async_smem();
            warp_arrive(ABAR(C::B_FULL + s));
            warp_arrive(ABAR(C::B_LEMPTY + sl));
          }
        }
      }
    } else if constexpr (KV == kKvPaged) {
      if (warp == 2) {
        for (int id = blockIdx.x; id < items && ok; id += step) {
          const AttendItem w = attend_item<KV>(p, id);
          for (int i = w.tiles.from; i < w.tiles.to && ok; ++i) {
            const int j0 = w.tiles.key(i);
            const uint32_t held = held_pages(p.pages, w.b, w.see, j0, lane);
            // values of rows that the window's or the sequence's edge leaves out
            const bool inner = (j0 + 128 <= w.see.sk || (j0 >= w.see.lo && j0 + 128 <= w.see.hi)) &&
                               held == (1u << (128 >> p.pages.log_page)) - 1u;
            for (int kv = 0; kv < 2; ++kv, ++use) {
              const int s = use % C::NS;
              ok = __all_sync(0xffffffffu, wait_bounded(ABAR(C::B_LAND + s), (use / C::NS) & 1, abort_flag));
              if (!ok) break;
              if (kv && !inner) {
                for (int r = lane; r < 128; r += 32) {
                  const int j = j0 + r;
                  const bool in = ((held >> (r >> p.pages.log_page)) & 1u) && (j < w.see.sk || (j >= w.see.lo && j < w.see.hi));
                  if (!in)
                    for (int pn = 0; pn < D / 64; ++pn)
#pragma unroll
                      for (int c = 0; c < 8; ++c)
                        *reinterpret_cast<uint4*>(base + C::OFF_RING + s * C::TILE + pn * 16384 + r * 128 + c * 16) =
                            make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
              }
              warp_arrive(ABAR(C::B_FULL + s));
            }
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------- softmax
    // The two warps of a row quarter leave together: every exit is agreed on at a pair barrier.
    const int hf = (warp - 4) >> 2, rt = threadIdx.x & 127, pair = 1 + (warp & 3);
    const int my_head = rt / p.rt.tokens, my_token = rt - my_head * p.rt.tokens;
    const uint32_t lrow = uint32_t((warp & 3) * 32) << 16;
    const uint32_t o_addr = tmem + lrow + C::O_COL + hf * (D / 2), q_addr = tmem + lrow + C::Q_COL + hf * (D / 4);
    float* xch = reinterpret_cast<float*>(base + C::OFF_X);
    float* scales = reinterpret_cast<float*>(base + C::OFF_SCALE) + (C::CODES ? (warp - 4) * 128 : 0);
    float sl2 = p.scale * 1.4426950408889634f, next_sl2 = sl2;
    // this thread's half of an item's query row (8 bits: in fp16, times a power of two)
    constexpr int QW = D / 4;  // 32-bit words
    auto load_queries = [&](const AttendItem& w, uint32_t (&q)[QW]) {
      const bool real = my_head < w.heads && w.t0 + my_token < w.nq;
      const uint4* src = reinterpret_cast<const uint4*>(p.Q + (size_t(w.head0 + (real ? my_head : 0)) * p.N + w.t0 + (real ? my_token : 0)) * D);
#pragma unroll
      for (int c = 0; c < QW / 4; ++c) {
        const uint4 x = real ? __ldg(src + hf * (QW / 4) + c) : make_uint4(0, 0, 0, 0);
        q[4 * c] = x.x;
        q[4 * c + 1] = x.y;
        q[4 * c + 2] = x.z;
        q[4 * c + 3] = x.w;
      }
      if constexpr (C::CODES) {
        uint32_t top = 0;  // over the whole row: both halves take the same factor
        for (int c = 0; c < QW / 2; ++c) {
          const uint4 x = real ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
          const uint32_t a[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) top = max(top, max(a[k] & 0x7fffu, (a[k] >> 16) & 0x7fffu));
        }
        const int field = min(253, 268 - int(top >> 7));  // top * 2^(field - 127) lies in [2^14, 2^15)
        const float f = top >= 0x7f80u ? __uint_as_float(0x7fc00000u) : exponent(field);  // infinity, NaN: NaN
        next_sl2 = p.scale * 1.4426950408889634f * exponent(254 - field);
#pragma unroll
        for (int k = 0; k < QW; ++k) q[k] = pack_f16x2(bf16_lo(q[k]) * f, bf16_hi(q[k]) * f);
      }
    };
    auto stage_queries = [&](const uint32_t (&q)[QW]) {
#pragma unroll
      for (int ch = 0; ch < QW / 16; ++ch) tmem_st16(q_addr + ch * 16, *reinterpret_cast<const uint32_t(*)[16]>(&q[ch * 16]));
      tmem_wait_st();
      tc_fence_before();
      warp_arrive(ABAR(C::B_Q));
    };
    bool ok = true, staged = false;
    int n = 0;  // key tiles so far
    uint32_t n_o = 0;
    for (int id = blockIdx.x; id < items && ok; id += step) {
      const AttendItem w = attend_item<KV>(p, id);
      if (!w.real) continue;
      const bool real = my_head < w.heads && w.t0 + my_token < w.nq;
      const int t = w.t0 + (real ? my_token : 0);
      const size_t row = size_t(w.head0 + (real ? my_head : 0)) * p.N + t;
      const int pos = w.n - w.nq + t;
      // the keys this row sees: up to z, and from a on or below the sinks' end
      const int z = max(-1, min(w.n - 1, pos + p.win.right)), a = max(0, pos - p.win.left);
      if (w.live() && !staged) {
        uint32_t q[QW];
        load_queries(w, q);
        stage_queries(q);
      }
      sl2 = next_sl2;
      staged = false;
      // 8 bits: a warp keeps its 64 keys' scales in shared memory (lanes 0-15 fetch K's, 16-31 V's),
      // the next tile's in registers
      float4 next_s;
      auto fetch_scales = [&](int i) {
        next_s = make_float4(0.f, 0.f, 0.f, 0.f);  // keys that nobody may see weigh nothing
        if (i >= w.tiles.to) return;
        const int j = w.tiles.key(i) + hf * 64 + 4 * (lane & 15);
        if (!w.see.any(j, 4)) return;
        const int page = p.pages.table[size_t(w.b) * p.pages.max_pages + (min(j, w.n - 1) >> p.pages.log_page)];
        if (page < 0 || page >= p.pages.num_pages) return;
        const size_t at = ((size_t(page) * p.Hkv + w.hk) << p.pages.log_page) + (j & ((1 << p.pages.log_page) - 1));
        next_s = __ldg(reinterpret_cast<const float4*>((lane < 16 ? p.pages.ks : p.pages.vs) + at));
        float* f = reinterpret_cast<float*>(&next_s);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (!(j + k < w.see.sk || (j + k >= w.see.lo && j + k < w.see.hi))) f[k] = 0.f;
      };
      if constexpr (C::CODES) {
        fetch_scales(w.tiles.from);
        __syncwarp();
      }
      float m = -INFINITY, l = 0.f;
      for (int i = w.tiles.from; i < w.tiles.to; ++i, ++n) {
        const int j0 = w.tiles.key(i) + hf * 64;  // of this half
        const uint32_t s_addr = tmem + lrow + C::S_COL + (n & 1) * 128 + hf * 64;
        uint32_t held = 0xffu;
        if constexpr (KV != kKvPlain) held = held_pages(p.pages, w.b, w.see, w.tiles.key(i), lane);
        const bool whole = j0 + 63 <= w.see.p0 + p.win.right && j0 + 64 <= w.n &&
                           (j0 >= w.see.p1 - p.win.left || j0 + 64 <= p.win.sinks) &&
                           (KV == kKvPlain || held == (1u << (128 >> p.pages.log_page)) - 1u);
        if constexpr (C::CODES) {
          __syncwarp();  // the previous tile's scales have been read
          reinterpret_cast<float4*>(scales)[lane] = next_s;
          __syncwarp();
          fetch_scales(i + 1);
          __syncwarp();
        }
        // the item's last tile: the next item's queries are fetched, and go to tensor memory once
        // these scores, the last that read the queries, are in
        uint32_t q[QW];
        bool stage_next = false;
        if (i + 1 == w.tiles.to && id + step < items) {
          const AttendItem x = attend_item<KV>(p, id + step);
          stage_next = x.live();
          if (stage_next) load_queries(x, q);
        }
        ok = __all_sync(0xffffffffu, wait_bounded(ABAR(C::B_S + (n & 1)), (n >> 1) & 1, abort_flag));
        tc_fence_after();
        uint32_t sc[64];
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) tmem_ld16(s_addr + ch * 16, *reinterpret_cast<uint32_t(*)[16]>(&sc[ch * 16]));
        if (stage_next && ok) {
          stage_queries(q);
          staged = true;
        }
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) tmem_wait_ld(*reinterpret_cast<uint32_t(*)[16]>(&sc[ch * 16]));
        if constexpr (C::CODES) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float4 f = reinterpret_cast<const float4*>(scales)[k];
            sc[4 * k] = __float_as_uint(__uint_as_float(sc[4 * k]) * f.x);
            sc[4 * k + 1] = __float_as_uint(__uint_as_float(sc[4 * k + 1]) * f.y);
            sc[4 * k + 2] = __float_as_uint(__uint_as_float(sc[4 * k + 2]) * f.z);
            sc[4 * k + 3] = __float_as_uint(__uint_as_float(sc[4 * k + 3]) * f.w);
          }
        }
        if (!whole) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t bits = ones_below(z - j0 + 1 - 32 * x) &
                            (~ones_below(a - j0 - 32 * x) | ones_below(p.win.sinks - j0 - 32 * x));
            if constexpr (KV != kKvPlain) {
              // 32 keys are one page of 32, a part of a larger one, or two of 16
              const int at = hf * 64 + 32 * x;
              if (p.pages.log_page >= 5) bits = ((held >> (at >> p.pages.log_page)) & 1u) ? bits : 0u;
              else bits &= ((held >> (at / 16)) & 1u ? 0xffffu : 0u) | ((held >> (at / 16 + 1)) & 1u ? 0xffff0000u : 0u);
            }
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (!((bits >> k) & 1u)) sc[32 * x + k] = __float_as_uint(-INFINITY);
          }
        }
        float mxp[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) mxp[k] = __uint_as_float(sc[k]);
#pragma unroll
        for (int k = 4; k < 60; k += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) mxp[e] = max3(mxp[e], __uint_as_float(sc[k + 2 * e]), __uint_as_float(sc[k + 2 * e + 1]));
#pragma unroll
        for (int e = 0; e < 4; ++e) mxp[e] = fmaxf(mxp[e], __uint_as_float(sc[60 + e]));
        float mx = fmaxf(fmaxf(mxp[0], mxp[1]), fmaxf(mxp[2], mxp[3])) * sl2;
        if (!pair_sync_and(pair, ok && !(mx > m + 8.f))) {
          xch[hf * 128 + rt] = mx;
          ok = pair_sync_and(pair, ok);
          if (!ok) break;
          mx = fmaxf(mx, xch[(hf ^ 1) * 128 + rt]);
          const bool grow = mx > m + 8.f, move = grow && m != -INFINITY;
          if (__any_sync(0xffffffffu, move)) {
            // O has to hold the products before this tile: V of tile n - 1 has been released
            ok = __all_sync(0xffffffffu, wait_bounded(ABAR(C::B_EMPTY + (2 * n - 1) % C::NS), ((2 * n - 1) / C::NS) & 1, abort_flag));
            tc_fence_after();
            const float f = move ? ex2(m - mx) : 1.f;
            rescale_row<D / 2>(o_addr, f);
            l *= f;
          }
          if (grow) m = mx;
          ok = pair_sync_and(pair, ok);
          if (!ok) break;
        }
        const float negm = m == -INFINITY ? 0.f : -m;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float e0 = __uint_as_float(sc[ch * 32 + 2 * k]), e1 = __uint_as_float(sc[ch * 32 + 2 * k + 1]);
            fma2(e0, e1, sl2, negm);
            e0 = ex2(e0);
            e1 = ex2(e1);
            add2(sum[2 * (k & 1)], sum[2 * (k & 1) + 1], e0, e1);
            if constexpr (C::CODES) {  // the value's scale may be NaN, or the weight huge beside it
              const float2 f = reinterpret_cast<const float2*>(scales + 64)[ch * 16 + k];
              pk[k] = pack_bf16x2(e0 * f.x, e1 * f.y);
            } else {
              pk[k] = pack_bf16x2_int(e0, e1);
            }
          }
          tmem_st16(s_addr + ch * 16, pk);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(ABAR(C::B_P + (n & 1)));
      }
      if (!ok) break;
      // both halves' sums, added in the same order on both sides
      xch[hf * 128 + rt] = l;
      if (w.live()) {
        ok = __all_sync(0xffffffffu, wait_bounded(ABAR(C::B_O), n_o, abort_flag));
        n_o ^= 1u;
      }
      ok = pair_sync_and(pair, ok);
      if (!ok) break;
      l = xch[rt] + xch[128 + rt];
      tc_fence_after();
      const float inv = l != 0.f ? 1.f / l : 0.f;  // l is NaN if a score was
      const size_t at = size_t(w.split) * size_t(p.B) * p.Hq * p.N + row;
#pragma unroll 1
      for (int ch = 0; ch < D / 64; ++ch) {
        __syncwarp();
        uint32_t o[2][16];
        if (w.live()) {
          tmem_ld16(o_addr + ch * 32, o[0]);
          tmem_ld16(o_addr + ch * 32 + 16, o[1]);
          tmem_wait_ld(o[0]);
          tmem_wait_ld(o[1]);
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) o[0][k] = o[1][k] = 0u;
        }
        const int c0 = hf * (D / 2) + ch * 32;
        if (p.splits > 1) store_part32(p.part + c0, real ? int64_t(at) * D : -1, o, inv);
        else store_rows32(p.O + c0, real ? int64_t(row) * D : -1, o, inv);
      }
      __syncwarp();
      if (real && hf == 0) {
        const float lg = l != 0.f ? m + __log2f(l) : -INFINITY;
        if (p.splits > 1) p.part_lse[at] = lg;
        else if (p.lse) p.lse[row] = lg * 0.6931471805599453f;
      }
      tc_fence_before();
      // the exchange's next words are written behind the next tile's vote, or behind this barrier
      if (!w.live()) ok = pair_sync_and(pair, ok);
    }
  }
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
#undef ABAR
}

// Joins the runs of a row: weights 2^(lse_s - max), in run order. One warp per row.
template <int D>
__global__ void __launch_bounds__(128) attend_join_kernel(const AttendTcParams p, int paged) {
  const int lane = threadIdx.x & 31;
  const int64_t rows = int64_t(p.B) * p.Hq * p.N, row = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= rows) return;
  if (paged) {
    const int b = int(row / (int64_t(p.Hq) * p.N)), t = int(row % p.N);
    if (t >= q_len_of(p.pages, b, p.N)) return;
  }
  float m = -INFINITY;
  for (int s = 0; s < p.splits; ++s) m = fmaxf(m, p.part_lse[s * rows + row]);
  const float m0 = m == -INFINITY ? 0.f : m;
  float l = 0.f, o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) o[i] = 0.f;
  for (int s = 0; s < p.splits; ++s) {
    const float w = tc::ex2(p.part_lse[s * rows + row] - m0);
    if (w == 0.f) continue;
    l += w;
    const float* src = p.part + (s * rows + row) * D;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = fmaf(w, src[i * 32 + lane], o[i]);
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) p.O[row * D + i * 32 + lane] = __float2bfloat16(o[i] * inv);
  if (lane == 0 && p.lse) p.lse[row] = l != 0.f ? (m0 + __log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace pisa
