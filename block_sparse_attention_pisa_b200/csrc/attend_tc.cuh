// Attention under a token-exact window on the tensor cores (tcgen05 / TMEM / TMA), over keys
// laid out plainly or in pages.
//
//   o = sum_j exp(s_j - m) v_j / l,  l = sum_j exp(s_j - m),  s_j = scale q.k_j, j visible
//
// one pass over the keys with a running maximum m and sum l per row.
//
// A persistent CTA per SM takes items in turn: two tiles (groups) of 128 rows of one key head
// that walk the 128-key tiles that some row of theirs sees (the tiles of the first tokens, then the
// window's); a group skips the ones that none of its rows sees. Warp roles:
//   warp 0       producer: K and V tiles by TMA (a page at a time in a paged cache) into a ring,
//                running ahead into the next item; it publishes which pages of a tile are held;
//   warp 1       issues every tcgen05.mma: per tile and group S = Q K^T (SS), then
//                O += P V (TS, P from tensor memory), the latter in two halves;
//   warp 3       loads the next item's queries once the last scores of this one are done;
//   warp 2       paged caches: clears the rows of a V tile that no row may see (unwritten rows
//                may hold anything, and 0 x NaN is NaN); 8 bits: warps 2-3 convert codes to bf16;
//   warps 4-11   softmax: one thread per row (group = warps 4-7 or 8-11), and the rows' output.
// Tensor memory: S of either group (128 columns each, P in bf16 over the first half of its own
// S) and O of either group (D columns each).
//
// The two groups alternate on the tensor core: while one group's exponentials run, the other's
// P V and next Q K^T do. A thread takes its whole row of S into registers, then hands P over in two
// halves, so that the product over the first 64 keys runs under the exponentials of the others.
// Products are issued by one lane and execute in order, so S of tile i + 1 may overwrite P of tile i
// behind the P V that reads it, and a group that sees its S(i + 1) (one commit) knows its O holds
// the products up to tile i: O is rescaled without a further wait. The accumulator is rescaled only
// when the maximum grows by more than 2^8.
//
// A value that is no finite number and that only some rows of its tile see would reach the others
// through a weight of zero. Looking at every such tile for it cost 5% (2 x 24 heads of 4096 x 128,
// 512 keys to either side: 156 us against 148); the rows' output is looked at instead. Items with a
// row that holds something that is no finite number are marked, and once the CTA is through it takes
// those again (a second pass of the same roles): such values leave the tiles that some row sees in
// part, and the rows that see them take them by themselves. No role of the first pass waits for it, and
// it costs a marked item what the first did, besides the search for the values (an infinity in the last
// tile of a causal head of 16384 x 128: 672 us, 248 without; of a million tokens: 297 ms, 280 without).
// It also holds its weights in a frame so far down that sums of the largest values stay in range: a
// weight may be 2^8 and there are many, so that the first pass leaves the range from values of about
// 2^120 on (and less, with many keys). What the first pass found finite stays, in full precision.
//
// Bound: at D = 128 a tile of 128 x 128 takes 2 x 512 cycles of tensor time, and a pair of tiles
// 2 x 512 x 2 = 2048, as long as its 2 x 16384 exponentials take at 16 per cycle. Measured, a pair
// takes about 4000: the softmax of two rows per scheduler 2300 (exponential 8 cycles per warp and
// instruction, the pack to bf16 as long again, two fma and add per value), and then, of either group,
// the chain "second half of P V, next Q K^T, its commit" that the other group only partly covers. Products
// and softmax of two groups could run beside each other in 2300; how the rest divides between that chain and
// the registers that spill (a whole row of S in flight: 156-180 bytes, 460 in 8 bits) is not measured.
// 2 x 24 heads of 4096 x 128, 512 keys to either side: 148-153 us by box, 0.64 PFLOP/s; 2 x 1024 tokens of
// 24 heads over a paged cache of 16 K, window 8192: 274 us, 0.76 PFLOP/s; causal, 16 and 4 heads of 32 K x
// 128: 4.1 ms, 1.07 PFLOP/s; D = 64 has the same softmax for half the products, and leaves 128 columns
// of tensor memory unused. What was tried and measured slower: one 128-row tile with two score buffers;
// two threads per row; a maximum guessed from the tile before; separate columns for P; packed fp32
// pairs for the scaling; setmaxnreg (the roles that give registers away spill); the last wave's pairs
// cut in two (one tile takes as long as a pair: its own chain; 151 us against 147).
// 8 bits, D = 64: 3 sequences of 333 tokens, 12 and 4 heads, 5 K keys: 62 us, all but about 10 (start and
// join) for the 14 tiles of an item in turn: 7000 cycles a pair, where the bf16 form takes 4000. At 67 us
// in all, it took 56 without the scales (128 products and 32 shared-memory loads of either kind per row
// and tile) and 65 without the conversion; the rest is not accounted for.
#pragma once

#include "attention_tc.cuh"
#include "window.cuh"

namespace pisa {

// A tile of 128 rows holds `tokens` consecutive tokens of all query heads of a key head (of up to
// 128 of them), head by head: row r is head r / tokens, token r % tokens. Shared keys are read once
// for all their heads, and a tile spans few positions. One box of a [heads][tokens][D] tensor
// map is such a tile; with a group that does not divide 128 a few rows stay idle (3 heads: 2).
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
  Pages pages;      // paged; of plain keys K and V alone, [B * Hkv][N][D]
  int B, Hq, Hkv, N;
  RowTiles rt;
  int G;            // query heads per key head
  int pairs;        // pairs of row tiles of a key head
  int part_pairs;   // of one part of its heads
  int splits;       // runs that a piece's tile list is cut into (plain keys: 1)
  int items;        // pairs * B * Hkv * splits
  long long patience;  // cycles that all of a CTA's items may take
  Window win;
  float scale;
};

template <int D, int KV>
struct AttendTcCfg {
  static constexpr int kThreads = 384;
  static constexpr bool CODES = KV == kKvPagedE4m3;
  static constexpr int TILE = 128 * D * 2;          // bytes of a 128-row bf16 tile
  static constexpr int NS = CODES ? 3 : (D == 128 ? 5 : 10);  // ring stages
  static constexpr int NL = CODES ? (D == 128 ? 3 : 6) : NS;  // landing stages (8 bits: tiles of codes)
  static constexpr int LAND = CODES ? 128 * D : 0;  // bytes of a landing stage of its own
  static constexpr int OFF_Q = 0;                   // two groups' queries
  static constexpr int OFF_RING = 2 * TILE;
  static constexpr int OFF_CODES = OFF_RING + NS * TILE;
  static constexpr int OFF_SCALE = OFF_CODES + NL * LAND;  // 8 bits: float [8 warps][K, V][128]
  static constexpr int B_FULL = 0;                  // [NS] stage holds its tile
  static constexpr int B_EMPTY = B_FULL + NS;       // [NS] products that read it are done (commit)
  static constexpr int B_LAND = B_EMPTY + NS;       // [NL] paged: V landed, not cleared yet; codes not converted yet
  static constexpr int B_LEMPTY = B_LAND + NL;      // [NL] 8 bits: codes converted (2 warps)
  static constexpr int B_Q = B_LEMPTY + NL;         // [2] a group's queries are in shared memory
  static constexpr int B_QEMPTY = B_Q + 2;          // [2] the item's last scores are done (commit)
  static constexpr int B_S = B_QEMPTY + 2;          // [2] S ready (commit)
  static constexpr int B_P = B_S + 2;               // [2] P written (4 warps)
  static constexpr int B_H = B_P + 2;               // [2] the first half of P written (4 warps)
  static constexpr int B_O = B_H + 2;               // [2] the item's last product is done (commit)
  static constexpr int B_END = B_O + 2;             // all products done (commit)
  static constexpr int NBARS = B_END + 1;
  static constexpr int OFF_BAR = OFF_SCALE + (CODES ? 8 * 2 * 128 * 4 : 0);
  static constexpr int OFF_MISC = OFF_BAR + 8 * NBARS;
  // Paged: bit i = page i of the tile is seen and held, for tile t at t % kHeld. Producer, converters
  // and softmax are at most 7 tiles apart.
  static constexpr int OFF_HELD = OFF_MISC + 16, kHeld = 16;
  // The items to take again: bit i of these words for the CTA's items i, i + 32 kMarks, ... (an item
  // that is taken again without need keeps what it has). Barriers of the second pass.
  static constexpr int OFF_MARKS = OFF_HELD + 4 * kHeld, kMarks = 32;
  static constexpr int OFF_BAR2 = OFF_MARKS + 4 * kMarks;
  static constexpr int SMEM = OFF_BAR2 + 8 * NBARS + 1024;
  static constexpr int S_COL = 0, O_COL = 256;
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
  // every row sees every key of [j0, j0 + 128)
  __device__ __forceinline__ bool all(const Window& w, int j0, int n) const {
    return j0 + 127 <= p0 + w.right && j0 + 128 <= n && (j0 >= p1 - w.left || j0 + 128 <= w.sinks);
  }
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
    const unsigned total = unsigned(ns + (w1 - w0));  // at most 2^23, times 148 runs
    from = 0;
    to = int(total);
    if (splits > 1) {
      from = int(total * unsigned(split) / unsigned(splits));
      to = int(total * unsigned(split + 1) / unsigned(splits));
    }
  }
  __device__ __forceinline__ int key(int i) const { return (i < ns ? i : first + i - ns) << 7; }
};

__device__ __forceinline__ uint32_t ones_below(int k) {  // bits [0, k) of a word, any k
  return k <= 0 ? 0u : (k >= 32 ? 0xffffffffu : (1u << k) - 1u);
}

// Paged: parity on B_LAND of the stage that use `u` (odd: V) takes; K goes straight to B_FULL.
template <int NS>
__device__ __forceinline__ uint32_t landed_parity(int u) {
  return uint32_t(NS % 2 ? u / (2 * NS) : u / NS) & 1u;
}

// bf16 values: any that is no finite number (an infinity or a NaN)
__device__ __forceinline__ bool any_not_finite(uint4 v) {
  constexpr uint32_t M = 0x7fff7fffu;
  const uint32_t top = __vmaxu2(__vmaxu2(v.x & M, v.y & M), __vmaxu2(v.z & M, v.w & M));
  return (top & 0x7f80u) == 0x7f80u || (top & 0x7f800000u) == 0x7f800000u;
}
// the low (high) half of a word as fp32 if it is no finite number, 0 if it is
__device__ __forceinline__ float not_finite_lo(uint32_t w) { return (w & 0x7f80u) == 0x7f80u ? __uint_as_float(w << 16) : 0.f; }
__device__ __forceinline__ float not_finite_hi(uint32_t w) {
  return (w & 0x7f800000u) == 0x7f800000u ? __uint_as_float(w & 0xffff0000u) : 0.f;
}
// two values with those that are no finite numbers as 0
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t w) {
  return ((w & 0x7f80u) == 0x7f80u ? 0u : w & 0xffffu) | ((w & 0x7f800000u) == 0x7f800000u ? 0u : w & 0xffff0000u);
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

// Wait of a warp for what may lie an item or more ahead (scores of a group that has no rows in the items
// before, the last scores over the item before): bounded by what all items may take, where other waits
// are bounded by about a second.
__device__ __forceinline__ bool wait_item(uint32_t bar, uint32_t parity, volatile int* abort_flag, long long patience) {
  bool ok = tc::mbar_try_wait(bar, parity);
  if (!ok) {
    const long long t0 = clock64();
    while (!(ok = tc::mbar_try_wait(bar, parity))) {
      if (*abort_flag) break;
      if (clock64() - t0 > tc::kWaitCycles + patience) {
        *abort_flag = 1;
        flag_error(kErrTimeout);
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
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

// fp32 pair: x = x * a + b
__device__ __forceinline__ void fma2(float& x0, float& x1, float a, float b) {
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmov.b64 z, {%3, %3};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+f"(x0), "+f"(x1)
      : "f"(a), "f"(b));
}
// the fp32 values of two words, times a and b
__device__ __forceinline__ void mul2(uint32_t& x0, uint32_t& x1, float a, float b) {
  asm("{\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "+r"(x0), "+r"(x1)
      : "f"(a), "f"(b));
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

// One piece of work: two tiles of a key head's rows over one run of their key tiles.
struct AttendItem {
  int b, hk, bh, split, n, nq;
  int t0[2], head0, heads;  // first token of either tile; first query head and how many are real
  Sight see[2], both;
  TileList tiles;
  bool real;
  // some row of a group that sees a part of [j0, j0 + 128) does not see all of it
  __device__ __forceinline__ bool edge(const Window& win, int j0) const {
    return (see[0].any(j0) && !see[0].all(win, j0, n)) || (see[1].any(j0) && !see[1].all(win, j0, n));
  }
};
// The CTA's items in turn: every gridDim.x-th, its coordinates kept by addition (a runtime division
// costs a role more than a hundred cycles, and there were six).
struct ItemWalk {
  int id, pair, split, hk, b;
  int d_pair, d_split, d_hk, d_b;
  __device__ __forceinline__ explicit ItemWalk(const AttendTcParams& p) {
    int x = blockIdx.x, y = gridDim.x;
    id = x;
    pair = x % p.pairs;
    d_pair = y % p.pairs;
    x /= p.pairs;
    y /= p.pairs;
    split = x % p.splits;
    d_split = y % p.splits;
    x /= p.splits;
    y /= p.splits;
    hk = x % p.Hkv;
    d_hk = y % p.Hkv;
    b = x / p.Hkv;
    d_b = y / p.Hkv;
  }
  __device__ __forceinline__ bool more(const AttendTcParams& p) const { return id < p.items; }
  __device__ __forceinline__ void advance(const AttendTcParams& p) {
    id += int(gridDim.x);
    pair += d_pair;
    split += d_split;
    hk += d_hk;
    b += d_b;
    if (pair >= p.pairs) pair -= p.pairs, ++split;
    if (split >= p.splits) split -= p.splits, ++hk;
    if (hk >= p.Hkv) hk -= p.Hkv, ++b;
  }
};
// The items of a pass: all of the CTA's, or in the second pass those that are marked.
template <bool AGAIN>
struct Items : ItemWalk {
  const uint32_t* marks;
  int i = 0;
  __device__ __forceinline__ Items(const AttendTcParams& p, const uint32_t* m) : ItemWalk(p), marks(m) { skip(p); }
  __device__ __forceinline__ void skip(const AttendTcParams& p) {
    if constexpr (AGAIN)
      while (more(p) && !((marks[(i >> 5) % AttendTcCfg<64, kKvPlain>::kMarks] >> (i & 31)) & 1u)) {
        ItemWalk::advance(p);
        ++i;
      }
  }
  __device__ __forceinline__ void advance(const AttendTcParams& p) {
    ItemWalk::advance(p);
    ++i;
    skip(p);
  }
};
// The item at `at` (which is one).
template <int KV>
__device__ __forceinline__ AttendItem attend_item(const AttendTcParams& p, const ItemWalk& at) {
  AttendItem w;
  w.split = at.split;
  w.b = at.b;
  w.hk = at.hk;
  w.bh = at.b * p.Hkv + at.hk;
  w.n = w.nq = p.N;
  if constexpr (KV != kKvPlain) {
    w.n = kv_len_of(p.pages, w.b);
    w.nq = q_len_of(p.pages, w.b, p.N);
  }
  int part = 0, pair = at.pair;
  if (p.rt.parts > 1) {
    part = pair / p.part_pairs;
    pair -= part * p.part_pairs;
  }
  pair = p.part_pairs - 1 - pair;  // causal: the rows with the most keys first
  w.head0 = w.b * p.Hq + w.hk * p.G + part * 128;
  w.heads = min(p.rt.heads, p.G - part * 128);
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    w.t0[g] = (2 * pair + g) * p.rt.tokens;
    if (w.t0[g] < w.nq) w.see[g].set(p.win, w.n - w.nq + w.t0[g], w.n - w.nq + min(w.t0[g] + p.rt.tokens, w.nq) - 1, w.n);
    else w.see[g].none();
  }
  w.real = w.t0[0] < w.nq;
  w.both = w.see[0];
  if (w.see[1].hi > 0) {
    w.both.lo = w.see[0].hi > 0 ? min(w.see[0].lo, w.see[1].lo) : w.see[1].lo;
    w.both.hi = max(w.see[0].hi, w.see[1].hi);
    w.both.sk = max(w.see[0].sk, w.see[1].sk);
  }
  w.tiles.set(w.both, w.split, p.splits);
  return w;
}

// Eight values of row `row` from column c on, as fp32.
template <int D, int KV>
__device__ __forceinline__ void load8(const void* x, const float* scales, int64_t row, int c, float (&v)[8]) {
  if constexpr (KV == kKvPagedE4m3) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(x) + row * D + c));
    const float f = __ldg(scales + row);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t two = e4m3x2_to_bf16x2((k < 2 ? w.x : w.y) >> (16 * (k & 1)));
      v[2 * k] = bf16_lo(two) * f;
      v[2 * k + 1] = bf16_hi(two) * f;
    }
  } else {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(static_cast<const bf16*>(x) + row * D + c));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = bf16_lo(u[k]);
      v[2 * k + 1] = bf16_hi(u[k]);
    }
  }
}

// The cache's row of key j of the item's sequence and key head (the plain one's), -1 if no page holds it.
template <int KV>
__device__ __forceinline__ int64_t row_of(const AttendTcParams& p, const AttendItem& w, int j) {
  if constexpr (KV == kKvPlain) return int64_t(w.bh) * p.N + j;
  const int page = p.pages.table[size_t(w.b) * p.pages.max_pages + (j >> p.pages.log_page)];
  if (page < 0 || page >= p.pages.num_pages) return -1;
  return ((int64_t(page) * p.Hkv + w.hk) << p.pages.log_page) + (j & ((1 << p.pages.log_page) - 1));
}

// A key (that a row sees) whose value is NaN throughout: the row is NaN by right.
template <int D, int KV>
__device__ __noinline__ bool lost_value(const AttendTcParams& p, const AttendItem& w, int j) {
  const int64_t at = row_of<KV>(p, w, j);
  bool nan = at >= 0;
#pragma unroll 1
  for (int c = 0; nan && c < D; c += 8) {
    float v[8];
    load8<D, KV>(p.pages.V, p.pages.vs, at, c, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) nan = nan && v[k] != v[k];
  }
  return nan;
}

// Output of the second pass, by a warp, a row per lane: the values that were left out of the tiles that
// some row sees in part join the rows that see them, and what the first pass left not finite is
// replaced (`inv` times the sums in tensor memory at `o_addr`; `to`: the row in O, or in the partial
// sums). A row sees keys up to z, and from a on or below the first tokens' end. Work: a search of
// the tiles for those seen in part (a lane per tile), and of those few (a lane per key).
template <int D, int KV>
__device__ __noinline__ void mend_rows(const AttendTcParams& p, const AttendItem& w, const Sight& mine, bool real, int z,
                                       int a, size_t to, uint32_t o_addr, float inv) {
  const int lane = threadIdx.x & 31;
  auto odd = [](float x) { return !(fabsf(x) < INFINITY); };
#pragma unroll 1
  for (int c = 0; c < D; c += 16) {
    uint32_t o[16];
    float x[16];
    __syncwarp();
    tc::tmem_ld16(o_addr + c, o);
    tc::tmem_wait_ld(o);
    bool open = false;  // a column that is NaN takes nothing any more
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      x[k] = __uint_as_float(o[k]) * inv;
      open |= x[k] == x[k];
    }
    if (__any_sync(0xffffffffu, real && open)) {
#pragma unroll 1
      for (int i0 = w.tiles.from; i0 < w.tiles.to; i0 += 32) {
        const int mine_i = w.tiles.key(i0 + lane);
        uint32_t tiles = __ballot_sync(0xffffffffu, i0 + lane < w.tiles.to && mine.any(mine_i) && w.edge(p.win, mine_i));
#pragma unroll 1
        for (; tiles; tiles &= tiles - 1)
#pragma unroll 1
          for (int s = 0; s < 128; s += 32) {
            const int j0 = w.tiles.key(i0 + __ffs(tiles) - 1) + s;
            // pages that no row sees are not looked up: their entries may hold anything
            const int64_t at = mine.any(j0 + lane, 1) ? row_of<KV>(p, w, j0 + lane) : -1;
            bool bad = false;
            float v[2][8];
            if (at >= 0) {
              load8<D, KV>(p.pages.V, p.pages.vs, at, c, v[0]);
              load8<D, KV>(p.pages.V, p.pages.vs, at, c + 8, v[1]);
#pragma unroll
              for (int k = 0; k < 16; ++k) bad |= odd(v[k >> 3][k & 7]);
            }
            uint32_t keys = __ballot_sync(0xffffffffu, bad);
#pragma unroll 1
            for (; keys; keys &= keys - 1) {
              const int j = j0 + __ffs(keys) - 1;
              const int64_t key = __shfl_sync(0xffffffffu, at, __ffs(keys) - 1);
              load8<D, KV>(p.pages.V, p.pages.vs, key, c, v[0]);
              load8<D, KV>(p.pages.V, p.pages.vs, key, c + 8, v[1]);
              const bool sees = j <= z && (j >= a || j < p.win.sinks);
#pragma unroll
              for (int k = 0; k < 16; ++k)
                if (sees && odd(v[k >> 3][k & 7])) x[k] += v[k >> 3][k & 7];
            }
          }
      }
    }
    if (!real) continue;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      if (KV != kKvPlain && p.splits > 1) {
        float* f = p.part + to * D + c + k;
        if (odd(*f)) *f = x[k];
      } else {
        bf16* f = p.O + to * D + c + k;
        if (odd(__bfloat162float(*f))) *f = __float2bfloat16(x[k]);
      }
    }
  }
}

// The roles of one pass over the CTA's items (AGAIN: the marked ones, see above). Counters of ring stages
// and barrier phases start with it: either pass has barriers of its own.
template <int D, int KV, bool AGAIN>
__device__ __forceinline__ void attend_pass(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                            const AttendTcParams& p, uint8_t* base, uint32_t base_u, uint32_t tmem) {
  using C = AttendTcCfg<D, KV>;
  using namespace tc;
  constexpr bool LANDS = KV == kKvPaged || (KV == kKvPlain && AGAIN);  // warp 2 goes over V's tiles
  volatile int* abort_flag = reinterpret_cast<int*>(base + C::OFF_MISC) + 1;
  uint32_t* held_mask = reinterpret_cast<uint32_t*>(base + C::OFF_HELD);
  uint32_t* marks = reinterpret_cast<uint32_t*>(base + C::OFF_MARKS);
  const uint32_t bar0 = base_u + (AGAIN ? C::OFF_BAR2 : C::OFF_BAR);
#define ABAR(i) (bar0 + 8u * uint32_t(i))
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (warp == 0) {
    // ------------------------------------------------------------- producer
    // Of an item's i-th tile, K is stage use 2 i and V 2 i + 1 behind the items before. Plain keys: lanes
    // 0 and 1 issue the two 64-column panels (D = 64: lane 0 alone). Pages: lane q looks page q of the
    // tile up (a tile ahead), and a copy per page and panel is issued by a lane of its own.
    bool ok = true;
    int use = 0;
    constexpr int NL = C::NL;  // the stages that the copies land in: the ring's, or those for codes
    for (Items<AGAIN> at(p, marks); at.more(p) && ok; at.advance(p)) {
      const AttendItem w = attend_item<KV>(p, at);
      if (!w.real) continue;
      const int per = 128 >> p.pages.log_page, size = 1 << p.pages.log_page;
      // pages that no row of the item sees, or that the table does not hold, stay out
      auto page_at = [&](int i) -> int {
        if (KV == kKvPlain || i >= w.tiles.to || lane >= per) return -1;
        const int j = w.tiles.key(i) + lane * size;
        return w.both.any(j, size) ? page_of(p.pages, w.b, j) : -1;
      };
      int ahead = page_at(w.tiles.from);
      for (int i = w.tiles.from; i < w.tiles.to && ok; ++i) {
        const int j0 = w.tiles.key(i);
        const int page = __shfl_sync(0xffffffffu, ahead, lane & (per - 1));
        const uint32_t held = __ballot_sync(0xffffffffu, ahead >= 0);
        ahead = page_at(i + 1);
        for (int kv = 0; kv < 2 && ok; ++kv, ++use) {
          const int s = use % NL;
          ok = __all_sync(0xffffffffu, wait_bounded(ABAR((C::CODES ? C::B_LEMPTY : C::B_EMPTY) + s), ((use / NL) & 1) ^ 1, abort_flag));
          if (!ok) break;
          const uint32_t dst = base_u + (C::CODES ? C::OFF_CODES + s * C::LAND : C::OFF_RING + s * C::TILE);
          const uint32_t bar = ABAR((C::CODES || (LANDS && kv) ? C::B_LAND : C::B_FULL) + s);
          if constexpr (KV == kKvPlain) {
            if (lane == 0) mbar_arrive_expect_tx(bar, C::TILE);
            __syncwarp();
            if (lane * 64 < D) tma_load_3d(dst + lane * 16384, kv ? &tmV : &tmK, bar, lane * 64, j0, w.bh);
          } else {
            if (lane == 0) {
              if (kv == 0) held_mask[(use >> 1) % C::kHeld] = held;
              mbar_arrive_expect_tx(bar, __popc(held) * size * D * (C::CODES ? 1 : 2));
            }
            __syncwarp();
            const int q = lane & (per - 1), panel = lane / per;  // whole rows of codes are one panel
            if (page >= 0 && panel < (C::CODES ? 1 : D / 64))
              tma_load_3d(dst + (C::CODES ? q * size * D : panel * 16384 + q * size * 128), kv ? &tmV : &tmK, bar,
                          panel * 64, 0, page * p.Hkv + w.hk);
          }
        }
      }
    }
    // no copy may still be in flight when the CTA exits
    if (lane == 0)
      for (int u = use > NL ? use - NL : 0; u < use; ++u) {
        if (LANDS && (u & 1)) wait_drain(ABAR(C::B_LAND + u % NL), landed_parity<NL>(u));
        else wait_drain(ABAR((C::CODES ? C::B_LAND : C::B_FULL) + u % NL), (u / NL) & 1);
      }
  } else if (warp == 1) {
    // ------------------------------------------------------------- products
    constexpr uint32_t idS = idesc_bf16(128, 128, false), idO = idesc_bf16(128, D, true);
    const bool lead = elect();
    bool ok = true;
    uint32_t n_p = 0, n_q = 0;  // bit g: phase of P, of the queries
    int use = 0;                // stage uses of the items before
    auto stage = [&](int u) { return base_u + C::OFF_RING + (u % C::NS) * C::TILE; };
    auto full = [&](int u) { return wait_warp(ABAR(C::B_FULL + u % C::NS), (u / C::NS) & 1, abort_flag); };
    Items<AGAIN> at(p, marks);
    AttendItem w = attend_item<KV>(p, at), next = w;  // the grid has no more CTAs than there are items, and a second pass has one
    while (at.more(p) && ok) {
      const int count = w.tiles.to - w.tiles.from;
      bool looked = false;
      if (w.real) {
        int last[2];  // a group's last tile of the run
        uint32_t before = 0, has_o = 0;  // bit g: it saw the tile before; its O holds a product of this item
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          last[g] = count - 1;
          while (last[g] >= 0 && !w.see[g].any(w.tiles.key(w.tiles.from + last[g]))) --last[g];
          if (w.see[g].hi > 0 && ok) ok = wait_warp(ABAR(C::B_Q + g), (n_q >> g) & 1u, abort_flag);
        }
        for (int i = -1; i < count && ok; ++i) {
          const bool more = i + 1 < count;
          const int jn = more ? w.tiles.key(w.tiles.from + i + 1) : 0;
          const uint64_t v = operand(stage(use + 2 * i + 1), 16384), k = operand(stage(use + 2 * i + 2), 16);
          uint32_t now = 0;
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const bool saw = (before >> g) & 1u;
            // the group has awaited V of this tile and K of the next before it signals P
            if (saw) {  // O += P V, by halves of the keys
              if (!(ok = wait_warp(ABAR(C::B_H + g), (n_p >> g) & 1u, abort_flag))) break;
              if (!(ok = full(use + 2 * i + 1))) break;
              tc_fence_after();
              if (lead) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  umma_ts(tmem + C::O_COL + g * D, tmem + C::S_COL + g * 128 + c * 8, v + c * (2048 >> 4), idO,
                          (((has_o >> g) & 1u) | uint32_t(c)) ? 1u : 0u);
              }
              if (!(ok = wait_warp(ABAR(C::B_P + g), (n_p >> g) & 1u, abort_flag))) break;
            }
            const bool sees = more && w.see[g].any(jn);
            if (sees && !(ok = full(use + 2 * i + 2))) break;
            tc_fence_after();
            if (lead) {
              if (saw) {  // O += P V
#pragma unroll
                for (int c = 4; c < 8; ++c)
                  umma_ts(tmem + C::O_COL + g * D, tmem + C::S_COL + g * 128 + c * 8, v + c * (2048 >> 4), idO, 1u);
                if (i == last[g]) umma_commit(ABAR(C::B_O + g));
              }
              if (sees) {  // S = Q K^T of the next tile
                const uint64_t q = operand(base_u + C::OFF_Q + g * C::TILE, 16);
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                  const uint32_t off = ((c >> 2) * 16384 + (c & 3) * 32) >> 4;
                  umma_ss(tmem + C::S_COL + g * 128, q + off, k + off, idS, c ? 1u : 0u);
                }
                umma_commit(ABAR(C::B_S + g));
              }
            }
            if (saw) {
              n_p ^= 1u << g;
              has_o |= 1u << g;
            }
            now |= uint32_t(sees) << g;
          }
          if (!ok) break;
          before = now;
          // a tile of the list is seen by one group at least, so its copies have been awaited
          if (lead) {
            if (i >= 0) umma_commit(ABAR(C::B_EMPTY + (use + 2 * i + 1) % C::NS));
            if (more) umma_commit(ABAR(C::B_EMPTY + (use + 2 * i + 2) % C::NS));
          }
          if (i + 2 >= count && !looked) {  // the run's last scores are issued: the queries may go
#pragma unroll
            for (int g = 0; g < 2; ++g)
              if (w.see[g].hi > 0) {
                if (lead) umma_commit(ABAR(C::B_QEMPTY + g));
                n_q ^= 1u << g;
              }
            at.advance(p);
            if (at.more(p)) next = attend_item<KV>(p, at);  // while the products run
            looked = true;
          }
        }
        use += 2 * count;
      }
      if (!looked) {
        at.advance(p);
        if (at.more(p)) next = attend_item<KV>(p, at);
      }
      w = next;
    }
    if (lead) {
      umma_commit(ABAR(C::B_END));
      wait_drain(ABAR(C::B_END), 0);  // nothing of ours may run on after the CTA frees TMEM
    }
    __syncwarp();
  } else if (warp < 4) {
    // ------------------------------------------------------------- queries; paged: rows nobody may see, codes
    bool ok = true;
    int use = 0;
    uint32_t n_q = 0, q_loaded = 0;  // bit g: phase of the queries, some were loaded
    for (Items<AGAIN> at(p, marks); at.more(p) && ok; at.advance(p)) {
      const AttendItem w = attend_item<KV>(p, at);
      if (!w.real) continue;
      const int count = w.tiles.to - w.tiles.from;
      if (warp == 3) {
        // the item's queries, once the last scores of the item before are done
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          if (w.see[g].hi == 0) continue;
          if (ok) ok = wait_item(ABAR(C::B_QEMPTY + g), ((n_q >> g) & 1u) ^ 1u, abort_flag, p.patience);
          if (ok && lane == 0) {
            mbar_arrive_expect_tx(ABAR(C::B_Q + g), p.rt.tokens * p.rt.heads * D * 2);
#pragma unroll
            for (int pn = 0; pn < D / 64; ++pn)
              tma_load_3d(base_u + C::OFF_Q + g * C::TILE + pn * 16384, &tmQ, ABAR(C::B_Q + g), pn * 64, w.t0[g], w.head0);
          }
          if (ok) {
            n_q ^= 1u << g;
            q_loaded |= 1u << g;
          }
        }
        if (!ok) break;
      }
      if constexpr (KV == kKvPagedE4m3) {
        // 16 codes per thread and step -> 32 bytes of the swizzled operand; rows that nobody may
        // see become zero. The scales stay out: scores and weights take them exactly in fp32. A
        // thread keeps its chunk of the rows and its row's place in the swizzle: steps are offsets.
        constexpr int CH = D / 16, STEP = 64 / CH;  // 16-code chunks of a row, rows of a step
        const int ct = threadIdx.x - 64, c = ct % CH, r0 = ct / CH, c0 = (2 * c) & 7;
        const uint32_t from = C::OFF_CODES + r0 * D + c * 16, to = C::OFF_RING + (c >> 2) * 16384 + r0 * 128;
        const uint32_t at_lo = (c0 ^ (r0 & 7)) << 4, at_hi = ((c0 + 1) ^ (r0 & 7)) << 4;
        for (int u = use; u < use + 2 * count; ++u) {
          const int sl = u % C::NL, s = u % C::NS, j0 = w.tiles.key(w.tiles.from + ((u - use) >> 1));
          ok = wait_bounded(ABAR(C::B_EMPTY + s), ((u / C::NS) & 1) ^ 1, abort_flag) &&
               wait_bounded(ABAR(C::B_LAND + sl), (u / C::NL) & 1, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          const uint32_t held = held_mask[(u >> 1) % C::kHeld];
          const bool inner = (j0 + 128 <= w.both.sk || (j0 >= w.both.lo && j0 + 128 <= w.both.hi)) &&
                             held == (1u << (128 >> p.pages.log_page)) - 1u;
          const uint8_t* src = base + from + sl * C::LAND;
          uint8_t* dst = base + to + s * C::TILE;
#pragma unroll 4
          for (int x = 0; x < 128 / STEP; ++x) {
            uint4 code = *reinterpret_cast<const uint4*>(src + x * STEP * D);
            if (!inner) {
              const int r = r0 + x * STEP, j = j0 + r;
              const bool in = ((held >> (r >> p.pages.log_page)) & 1u) && (j < w.both.sk || (j >= w.both.lo && j < w.both.hi));
              if (!in) code = make_uint4(0, 0, 0, 0);
            }
            *reinterpret_cast<uint4*>(dst + x * STEP * 128 + at_lo) =
                make_uint4(e4m3x2_to_bf16x2(code.x), e4m3x2_to_bf16x2(code.x >> 16), e4m3x2_to_bf16x2(code.y),
                           e4m3x2_to_bf16x2(code.y >> 16));
            *reinterpret_cast<uint4*>(dst + x * STEP * 128 + at_hi) =
                make_uint4(e4m3x2_to_bf16x2(code.z), e4m3x2_to_bf16x2(code.z >> 16), e4m3x2_to_bf16x2(code.w),
                           e4m3x2_to_bf16x2(code.w >> 16));
          }
          fence_proxy_async_smem();
          warp_arrive(ABAR(C::B_FULL + s));
          warp_arrive(ABAR(C::B_LEMPTY + sl));
        }
      } else if constexpr (LANDS) {
        if (warp == 2) {
          for (int u = use + 1; u < use + 2 * count; u += 2) {
            const int s = u % C::NS, j0 = w.tiles.key(w.tiles.from + ((u - use) >> 1));
            ok = __all_sync(0xffffffffu, wait_bounded(ABAR(C::B_LAND + s), landed_parity<C::NS>(u), abort_flag));
            if (!ok) break;
            const uint32_t held = KV == kKvPaged ? held_mask[(u >> 1) % C::kHeld] : 0u;
            // values of rows that the window's or the sequence's edge leaves out
            const bool inner = j0 + 128 <= w.both.sk || (j0 >= w.both.lo && j0 + 128 <= w.both.hi);
            if (KV == kKvPaged && !(inner && held == (1u << (128 >> p.pages.log_page)) - 1u)) {
              for (int r = lane; r < 128; r += 32) {
                const int j = j0 + r;
                const bool in = ((held >> (r >> p.pages.log_page)) & 1u) && (j < w.both.sk || (j >= w.both.lo && j < w.both.hi));
                if (!in)
                  for (int pn = 0; pn < D / 64; ++pn)
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                      *reinterpret_cast<uint4*>(base + C::OFF_RING + s * C::TILE + pn * 16384 + r * 128 + c * 16) =
                          make_uint4(0, 0, 0, 0);
              }
              fence_proxy_async_smem();
            }
            if (AGAIN && w.edge(p.win, j0)) {  // values that are no finite numbers: mend_rows adds them
#pragma unroll 1
              for (int x = lane; x < C::TILE / 16; x += 32) {
                uint4* v = reinterpret_cast<uint4*>(base + C::OFF_RING + s * C::TILE) + x;
                if (any_not_finite(*v))
                  *v = make_uint4(finite_or_zero(v->x), finite_or_zero(v->y), finite_or_zero(v->z), finite_or_zero(v->w));
              }
              fence_proxy_async_smem();
            }
            warp_arrive(ABAR(C::B_FULL + s));
          }
        }
      }
      use += 2 * count;
    }
    // no copy may still be in flight when the CTA exits
    if (lane == 0)
      for (int g = 0; g < 2; ++g)
        if ((q_loaded >> g) & 1u) wait_drain(ABAR(C::B_Q + g), ((n_q >> g) & 1u) ^ 1u);
  } else {
    // ------------------------------------------------------------- softmax
    const int g = (warp - 4) >> 2;
    const int my_head = int(threadIdx.x & 127) / p.rt.tokens, my_token = int(threadIdx.x & 127) - my_head * p.rt.tokens;
    const uint32_t lrow = uint32_t((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + lrow + C::S_COL + g * 128, o_addr = tmem + lrow + C::O_COL + g * D;
    const float sl2 = p.scale * 1.4426950408889634f;
    float* scales = reinterpret_cast<float*>(base + C::OFF_SCALE) + (C::CODES ? (warp - 4) * 256 : 0);
    const uint32_t full_mask = (1u << (128 >> p.pages.log_page)) - 1u;
    bool ok = true;
    uint32_t n_s = 0, n_o = 0;
    int use = 0;  // stage uses of the items before
    for (Items<AGAIN> at(p, marks); at.more(p) && ok; at.advance(p)) {
      const AttendItem w = attend_item<KV>(p, at);
      if (!w.real) continue;
      const Sight mine = g ? w.see[1] : w.see[0];
      const int t0 = g ? w.t0[1] : w.t0[0];
      const bool real = my_head < w.heads && t0 + my_token < w.nq;
      const int t = t0 + (real ? my_token : 0);
      const size_t row = size_t(w.head0 + (real ? my_head : 0)) * p.N + t;
      const int pos = w.n - w.nq + t;
      // the keys this row sees: up to z, and from a on or below the sinks' end
      const int z = max(-1, min(w.n - 1, pos + p.win.right)), a = max(0, pos - p.win.left);
      // 8 bits: a warp keeps its tile's scales in shared memory, the next tile's in registers
      float4 next_k, next_v;
      auto fetch_scales = [&](int i) {
        next_k = next_v = make_float4(0.f, 0.f, 0.f, 0.f);  // keys that nobody may see weigh nothing
        while (i < w.tiles.to && !mine.any(w.tiles.key(i))) ++i;
        if (i >= w.tiles.to) return;
        const int j = w.tiles.key(i) + 4 * lane;
        const int page = p.pages.table[size_t(w.b) * p.pages.max_pages + (min(j, w.n - 1) >> p.pages.log_page)];
        const bool in = mine.any(j, 4) && page >= 0 && page < p.pages.num_pages;
        if (!in) return;
        const size_t at = ((size_t(page) * p.Hkv + w.hk) << p.pages.log_page) + (j & ((1 << p.pages.log_page) - 1));
        next_k = __ldg(reinterpret_cast<const float4*>(p.pages.ks + at));
        next_v = __ldg(reinterpret_cast<const float4*>(p.pages.vs + at));
        float* f = reinterpret_cast<float*>(&next_v);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (!(j + k < mine.sk || (j + k >= mine.lo && j + k < mine.hi)) ||
              (AGAIN && !(fabsf(f[k]) < INFINITY) && w.edge(p.win, w.tiles.key(i))))
            f[k] = 0.f;
      };
      if constexpr (C::CODES) fetch_scales(w.tiles.from);
      // second pass: 2^-c times a weight, so that the run's weights (2^8 at most) sum to no more than one
      const int c = AGAIN ? 40 - __clz(max(1, w.tiles.to - w.tiles.from) * 128 - 1) : 0;
      const float frame = exponent(127 - c);
      float m = -INFINITY, l = 0.f;
      uint32_t done = 0;
      for (int i = w.tiles.from; i < w.tiles.to; ++i) {
        const int j0 = w.tiles.key(i);
        if (!mine.any(j0)) continue;
        const bool seen = mine.all(p.win, j0, w.n);
        if constexpr (C::CODES) {
          __syncwarp();  // the previous tile's scales have been read
          reinterpret_cast<float4*>(scales)[lane] = next_k;
          reinterpret_cast<float4*>(scales + 128)[lane] = next_v;
          __syncwarp();
          fetch_scales(i + 1);
          __syncwarp();
        }
        ok = wait_item(ABAR(C::B_S + g), n_s, abort_flag, p.patience);
        if (!ok) break;
        n_s ^= 1u;
        tc_fence_after();
        uint32_t held = 0xffu;
        if constexpr (KV != kKvPlain) held = held_mask[((use >> 1) + i - w.tiles.from) % C::kHeld];
        const bool whole = seen && (KV == kKvPlain || held == full_mask);
        uint32_t sc[128];
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) tmem_ld16(s_addr + ch * 16, *reinterpret_cast<uint32_t(*)[16]>(&sc[ch * 16]));
#pragma unroll
        for (int ch = 0; ch < 8; ++ch) tmem_wait_ld(*reinterpret_cast<uint32_t(*)[16]>(&sc[ch * 16]));
        if constexpr (C::CODES) {
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const float4 f = reinterpret_cast<const float4*>(scales)[k];
            mul2(sc[4 * k], sc[4 * k + 1], f.x, f.y);
            mul2(sc[4 * k + 2], sc[4 * k + 3], f.z, f.w);
          }
        }
        if (!whole) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t bits = ones_below(z - j0 + 1 - 32 * x) &
                            (~ones_below(a - j0 - 32 * x) | ones_below(p.win.sinks - j0 - 32 * x));
            if constexpr (KV != kKvPlain) {
              // 32 keys are one page of 32, a part of a larger one, or two of 16
              if (p.pages.log_page >= 5) bits = ((held >> ((32 * x) >> p.pages.log_page)) & 1u) ? bits : 0u;
              else bits &= ((held >> (2 * x)) & 1u ? 0xffffu : 0u) | ((held >> (2 * x + 1)) & 1u ? 0xffff0000u : 0u);
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
        for (int k = 4; k < 124; k += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) mxp[e] = max3(mxp[e], __uint_as_float(sc[k + 2 * e]), __uint_as_float(sc[k + 2 * e + 1]));
#pragma unroll
        for (int e = 0; e < 4; ++e) mxp[e] = fmaxf(mxp[e], __uint_as_float(sc[124 + e]));
        const float mx = fmaxf(fmaxf(mxp[0], mxp[1]), fmaxf(mxp[2], mxp[3])) * sl2;
        const bool grow = mx > m + 8.f;
        const bool move = grow && m != -INFINITY;
        if (__any_sync(0xffffffffu, move)) {  // S(i) is behind every earlier product of the group
          const float f = move ? ex2(m - mx) : 1.f;
          rescale_row<D>(o_addr, f);
          l *= f;
        }
        if (grow) m = mx;
        const float negm = m == -INFINITY ? 0.f : -m;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t pk[16];
          float4 f;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float e0 = ex2(fmaf(__uint_as_float(sc[ch * 32 + 2 * k]), sl2, negm));
            const float e1 = ex2(fmaf(__uint_as_float(sc[ch * 32 + 2 * k + 1]), sl2, negm));
            sum[k & 3] += e0 + e1;
            if constexpr (C::CODES) {  // the value's scale may be NaN, or the weight huge beside it
              if (k % 2 == 0) f = reinterpret_cast<const float4*>(scales + 128)[ch * 8 + k / 2];
              uint32_t x0 = __float_as_uint(AGAIN ? e0 * frame : e0), x1 = __float_as_uint(AGAIN ? e1 * frame : e1);
              mul2(x0, x1, k % 2 ? f.z : f.x, k % 2 ? f.w : f.y);
              pk[k] = pack_bf16x2(__uint_as_float(x0), __uint_as_float(x1));
            } else {
              pk[k] = AGAIN ? pack_bf16x2(e0 * frame, e1 * frame) : pack_bf16x2(e0, e1);
            }
          }
          tmem_st16(s_addr + ch * 16, pk);
          if (ch == 1) {
            tmem_wait_st();
            tc_fence_before();
            warp_arrive(ABAR(C::B_H + g));
          }
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(ABAR(C::B_P + g));
        done = 1;
      }
      if (ok && done) {
        ok = __all_sync(0xffffffffu, wait_bounded(ABAR(C::B_O + g), n_o, abort_flag));
        n_o ^= 1u;
      }
      if (!ok) break;
      tc_fence_after();
      const float inv = l != 0.f ? 1.f / l : 0.f;  // l is NaN if a score was
      const bool split_out = KV != kKvPlain && p.splits > 1;
      const size_t to = size_t(w.split) * size_t(p.B) * p.Hq * p.N + row;
      if constexpr (AGAIN) {
        if (done) mend_rows<D, KV>(p, w, mine, real, z, a, split_out ? to : row, o_addr, inv * exponent(127 + c));
        tc_fence_before();
        use += 2 * (w.tiles.to - w.tiles.from);
        continue;
      }
      float zero[2] = {0.f, 0.f};  // NaN once a value is no finite number
#pragma unroll 1
      for (int ch = 0; ch < D / 32; ++ch) {
        __syncwarp();
        uint32_t o[2][16];
        if (done) {
          tmem_ld16(o_addr + ch * 32, o[0]);
          tmem_ld16(o_addr + ch * 32 + 16, o[1]);
          tmem_wait_ld(o[0]);
          tmem_wait_ld(o[1]);
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) o[0][k] = o[1][k] = 0u;
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          zero[0] = fmaf(__uint_as_float(o[0][k]), 0.f, zero[0]);
          zero[1] = fmaf(__uint_as_float(o[1][k]), 0.f, zero[1]);
        }
        if (split_out) store_part32(p.part + ch * 32, real ? int64_t(to) * D : -1, o, inv);
        else store_rows32(p.O + ch * 32, real ? int64_t(row) * D : -1, o, inv);
      }
      __syncwarp();
      if (real) {
        const float lg = l != 0.f ? m + __log2f(l) : -INFINITY;
        if (split_out) p.part_lse[to] = lg;
        else if (p.lse) p.lse[row] = lg * 0.6931471805599453f;
      }
      const bool odd = real && done && zero[0] + zero[1] != 0.f && l == l;
      // a row whose own value is lost is left alone: in a sequence that is lost from a token on, few items are marked
      if (__any_sync(0xffffffffu, odd && !(pos >= 0 && pos <= z && lost_value<D, KV>(p, w, pos))) && lane == 0) {
        const uint32_t item = uint32_t(at.id) / gridDim.x;
        atomicOr(marks + (item >> 5) % C::kMarks, 1u << (item & 31));
        reinterpret_cast<volatile int*>(base + C::OFF_MISC)[2] = 1;
      }
      tc_fence_before();
      use += 2 * (w.tiles.to - w.tiles.from);
    }
  }
#undef ABAR
}

// The second pass: rare, and out of line so that the first pass keeps its registers.
template <int D, int KV>
__device__ __noinline__ void attend_again(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                                          const AttendTcParams& p, uint8_t* base, uint32_t base_u, uint32_t tmem) {
  attend_pass<D, KV, true>(tmQ, tmK, tmV, p, base, base_u, tmem);
}

template <class C>
__device__ __forceinline__ void init_barriers(uint32_t bar0) {
  using tc::mbar_init;
#define ABAR(i) (bar0 + 8u * uint32_t(i))
  for (int s = 0; s < C::NS; ++s) {
    mbar_init(ABAR(C::B_FULL + s), C::CODES ? 2 : 1);
    mbar_init(ABAR(C::B_EMPTY + s), 1);
  }
  for (int s = 0; s < C::NL; ++s) {
    mbar_init(ABAR(C::B_LAND + s), 1);
    mbar_init(ABAR(C::B_LEMPTY + s), 2);
  }
  for (int g = 0; g < 2; ++g) {
    mbar_init(ABAR(C::B_Q + g), 1);
    mbar_init(ABAR(C::B_QEMPTY + g), 1);
    mbar_init(ABAR(C::B_S + g), 1);
    mbar_init(ABAR(C::B_P + g), 4);
    mbar_init(ABAR(C::B_H + g), 4);
    mbar_init(ABAR(C::B_O + g), 1);
  }
  mbar_init(ABAR(C::B_END), 1);
  tc::mbar_init_fence();
#undef ABAR
}

template <int D, int KV>
__global__ void __launch_bounds__(384, 1)
attend_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, const __grid_constant__ AttendTcParams p) {
  using C = AttendTcCfg<D, KV>;
  using namespace tc;
  extern __shared__ __align__(16) uint8_t attend_smem[];
  const uint32_t raw_u = smem_u32(attend_smem);
  const uint32_t base_u = (raw_u + 1023u) & ~1023u;
  uint8_t* base = attend_smem + (base_u - raw_u);
  volatile int* misc = reinterpret_cast<int*>(base + C::OFF_MISC);  // tensor memory, abort flag, items to take again
  asm volatile("griddepcontrol.launch_dependents;");
  const int warp = threadIdx.x >> 5;

  if (threadIdx.x == 0) {
    misc[1] = misc[2] = 0;
    init_barriers<C>(base_u + C::OFF_BAR);
  }
  if (warp == 2) {
    tmem_alloc(base_u + C::OFF_MISC, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  if (warp == 3) reinterpret_cast<uint32_t*>(base + C::OFF_MARKS)[threadIdx.x & 31] = 0;
  static_assert(C::kMarks == 32, "a lane per word");
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uint32_t(misc[0]);
  attend_pass<D, KV, false>(tmQ, tmK, tmV, p, base, base_u, tmem);
  __syncthreads();
  if (misc[2] && !misc[1]) {
    tc_fence_after();
    if (threadIdx.x == 0) init_barriers<C>(base_u + C::OFF_BAR2);
    __syncthreads();
    attend_again<D, KV>(tmQ, tmK, tmV, p, base, base_u, tmem);
    __syncthreads();
  }
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the runs of a row: weights 2^(lse_s - max), in run order. D / 4 lanes per row, whose loads of
// several runs are in flight at once. Bound by memory (the partial sums are read once). The sum of the
// runs (no more than 148) is held 2^8 below its size, in range for any results of theirs.
constexpr int kJoinThreads = 256;
// Its blocks may start while the partial sums are still written: no loads through the read-only path.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(const AttendTcParams p) {
  constexpr int LANES = D / 4, ROWS = kJoinThreads / LANES;
  const int64_t rows = int64_t(p.B) * p.Hq * p.N, row = int64_t(blockIdx.x) * ROWS + threadIdx.x / LANES;
  const int c = threadIdx.x % LANES * 4;
  // every block waits, so that this grid does not end before the one it depends on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (row >= rows) return;
  const int b = int(row / (int64_t(p.Hq) * p.N)), t = int(row % p.N);
  if (t >= q_len_of(p.pages, b, p.N)) return;
  float m = -INFINITY;
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s) m = fmaxf(m, __ldcg(p.part_lse + s * rows + row));
  const float m0 = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = 0; s < p.splits; ++s) {  // a run that saw nothing holds zeros
    const float w = tc::ex2(__ldcg(p.part_lse + s * rows + row) - m0) * exponent(127 - 8);
    const float4 x = __ldcs(reinterpret_cast<const float4*>(p.part + (s * rows + row) * D + c));
    l += w;
    o = make_float4(fmaf(w, x.x, o.x), fmaf(w, x.y, o.y), fmaf(w, x.z, o.z), fmaf(w, x.w, o.w));
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  *reinterpret_cast<uint2*>(p.O + row * D + c) = make_uint2(pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
  if (c == 0 && p.lse) p.lse[row] = l != 0.f ? (m0 + __log2f(l * exponent(127 + 8))) * 0.6931471805599453f : -INFINITY;
}

}  // namespace pisa
