// Window mask and page addressing shared by the windowed attention, its gradient and the
// paged cache kernels.
//
// A query at position p sees key j of its sequence if
//   j <= p + right  and  (j >= p - left  or  j < sinks),
// so the keys a run of queries [p0, p1] can see are two ranges: the first tokens
// [0, min(sinks, hi)) and the window [max(0, p0 - left), hi) with hi = min(n, p1 + right + 1).
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace pisa {

constexpr int kMaxTokens = 1 << 30;  // positions, window reaches and sinks stay below: sums fit 32 bits

struct Window {
  int left, right, sinks;  // below kMaxTokens; kMaxTokens - 1 stands for no limit
};

enum { kKvPlain = 0, kKvPaged = 1, kKvPagedE4m3 = 2 };

// Pages of tokens: K, V [num_pages][Hkv][page][D], scales [num_pages][Hkv][page] (8 bits only).
struct Pages {
  const void* K;
  const void* V;
  const float* ks;
  const float* vs;
  const int32_t* table;  // [B][max_pages]
  const int32_t* kv_lens;
  const int32_t* q_lens;  // may be null: every sequence has N new tokens
  int num_pages, max_pages, log_page;
};

// Lengths are device data: what lies outside [0, capacity] (or [0, N]) is flagged and clamped.
__device__ __forceinline__ int checked_len(int n, int most) {
  if (n >= 0 && n <= most) return n;
  flag_error(kErrBadIndex);
  return n < 0 ? 0 : most;
}
__device__ __forceinline__ int kv_len_of(const Pages& g, int b) {
  return checked_len(g.kv_lens[b], g.max_pages << g.log_page);
}
__device__ __forceinline__ int q_len_of(const Pages& g, int b, int N) {
  return g.q_lens ? checked_len(g.q_lens[b], N) : N;
}
// Page that holds position `pos` of sequence b, or -1 (flagged) if the table has none there.
__device__ __forceinline__ int page_of(const Pages& g, int b, int pos) {
  const int at = g.table[size_t(b) * g.max_pages + (pos >> g.log_page)];
  if (at >= 0 && at < g.num_pages) return at;
  flag_error(kErrBadIndex);
  return -1;
}

// two e4m3 codes (low byte first) -> two bf16, exact. An e4m3 code seeeemmm placed as the
// bf16 bits s0000eee emmm0000 is its value times 2^-120 (the biases differ by 127 - 7), also
// for subnormal codes: one exact product restores it. S.1111.111 is NaN in e4m3 and would
// read as 480: it is put back by the caller's scale (a row that holds a NaN has scale NaN).
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t two) {
  uint32_t w = __byte_perm(two, 0, 0x1404);              // bytes into the high halves: lo<<8, hi<<24
  w = (w & 0x80008000u) | ((w & 0x7f007f00u) >> 4);
  const uint32_t up = 0x7b807b80u;                        // 2^120 twice
  __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162*>(&w), *reinterpret_cast<const __nv_bfloat162*>(&up));
  return *reinterpret_cast<uint32_t*>(&r);
}

// the power of two with these bits in its fp32 exponent field
__device__ __forceinline__ float exponent(int field) { return __uint_as_float(uint32_t(field) << 23); }

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
}  // namespace pisa
