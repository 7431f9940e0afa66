// C ABI of the windowed attention, its gradient, the paged cache and the attention over it:
// argument checks and launches. Included once by pisa_api.cu, whose helpers it uses.
#pragma once

namespace {

pisa_status_t check_aligned(const void* p, const char* name, unsigned align) {
  if (p == nullptr) return fail(PISA_ERR_INVALID_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) & (align - 1u))
    return fail(PISA_ERR_INVALID_ARG, "%s is not %u-byte aligned", name, align);
  return ok();
}

pisa_status_t check_scale(float scale) {
  if (!std::isfinite(scale) || !(scale > 0.f))
    return fail(PISA_ERR_INVALID_ARG, "scale=%g (must be finite and > 0)", double(scale));
  return ok();
}

// Heads, tokens and rows of any of these calls. Sets *empty if there is nothing to do.
pisa_status_t check_heads(int64_t B, int64_t Hq, int64_t Hkv, int64_t N, int32_t d, bool* empty) {
  *empty = false;
  if (B < 0 || Hq < 0 || Hkv < 0 || N < 0)
    return fail(PISA_ERR_INVALID_ARG, "negative shape (B=%lld Hq=%lld Hkv=%lld N=%lld)", (long long)B, (long long)Hq,
                (long long)Hkv, (long long)N);
  if (d <= 0) return fail(PISA_ERR_INVALID_ARG, "d must be positive (d=%d)", d);
  if (B == 0 || Hq == 0 || N == 0) {
    *empty = true;
    return ok();
  }
  if (Hkv == 0 || Hq % Hkv != 0)
    return fail(PISA_ERR_INVALID_ARG, "Hq=%lld is not a multiple of Hkv=%lld", (long long)Hq, (long long)Hkv);
  if (d != 64 && d != 128) return fail(PISA_ERR_UNSUPPORTED, "head dimension d=%d (supported: 64, 128)", d);
  if (N > pisa::kMaxTokens) return fail(PISA_ERR_UNSUPPORTED, "N=%lld exceeds %d", (long long)N, pisa::kMaxTokens);
  // B * Hq * N < 2^31 without overflow: each factor is below 2^31
  if (B * Hq > INT32_MAX || B * Hq * N > INT32_MAX)
    return fail(PISA_ERR_UNSUPPORTED, "B*Hq*N exceeds 2^31 - 1 rows");
  return ok();
}

pisa_status_t check_window(const pisa_window_t& w, pisa::Window* out) {
  if (w.left < -1 || w.right < -1 || w.sinks < 0)
    return fail(PISA_ERR_INVALID_ARG, "window left=%d right=%d (must be >= -1) sinks=%d (must be >= 0)", w.left,
                w.right, w.sinks);
  const auto reach = [](int32_t x) { return x < 0 || x >= pisa::kMaxTokens ? pisa::kMaxTokens - 1 : x; };
  *out = pisa::Window{reach(w.left), reach(w.right), reach(w.sinks)};
  return ok();
}

pisa_status_t check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return ok();
  PISA_TRY(check_aligned(ws, "workspace", 256));
  if (have < need) return fail(PISA_ERR_INVALID_ARG, "workspace holds %zu bytes, %zu are needed", have, need);
  return ok();
}

pisa_status_t check_cache(const pisa_cache_t& c, const pisa_sequences_t& s, int32_t Hq, bool* empty, pisa::Pages* g) {
  PISA_TRY(check_heads(s.B, Hq, c.Hkv, s.N, c.d, empty));
  if (*empty) return ok();
  if (c.type != PISA_CACHE_BF16 && c.type != PISA_CACHE_E4M3)
    return fail(PISA_ERR_INVALID_ARG, "cache type=%d (must be PISA_CACHE_BF16 or PISA_CACHE_E4M3)", c.type);
  if (c.page <= 0 || c.num_pages <= 0 || s.max_pages <= 0)
    return fail(PISA_ERR_INVALID_ARG, "page=%d num_pages=%d max_pages=%d (must be positive)", c.page, c.num_pages,
                s.max_pages);
  if (c.page != 16 && c.page != 32 && c.page != 64 && c.page != 128)
    return fail(PISA_ERR_UNSUPPORTED, "page=%d (supported: 16, 32, 64, 128)", c.page);
  if (int64_t(s.max_pages) * c.page > pisa::kMaxTokens)
    return fail(PISA_ERR_UNSUPPORTED, "max_pages*page exceeds %d tokens", pisa::kMaxTokens);
  if (int64_t(c.num_pages) * c.Hkv > INT32_MAX)
    return fail(PISA_ERR_UNSUPPORTED, "num_pages*Hkv exceeds 2^31 - 1");
  PISA_TRY(check_ptr(c.K, "cache K"));
  PISA_TRY(check_ptr(c.V, "cache V"));
  if (c.type == PISA_CACHE_E4M3) {
    PISA_TRY(check_ptr(c.k_scale, "k_scale"));
    PISA_TRY(check_ptr(c.v_scale, "v_scale"));
  }
  PISA_TRY(check_aligned(s.page_table, "page_table", 4));
  PISA_TRY(check_aligned(s.kv_lens, "kv_lens", 4));
  if (s.q_lens != nullptr) PISA_TRY(check_aligned(s.q_lens, "q_lens", 4));
  int log_page = 4;
  while ((1 << log_page) < c.page) ++log_page;
  *g = pisa::Pages{c.K, c.V, c.k_scale, c.v_scale, s.page_table, s.kv_lens, s.q_lens, c.num_pages, s.max_pages, log_page};
  return ok();
}

// the paged cache's kernels: `values` of a row per thread, rows dealt out to the CTAs in turn
template <typename Kernel>
pisa_status_t launch_cache(Kernel k, const pisa::CacheParams& p, int d, int values, int sms, cudaStream_t st,
                           const char* what) {
  const int64_t per = int64_t(pisa::kCacheThreads) * values / d;
  const int64_t ctas = (p.rows + per - 1) / per;
  const int64_t most = int64_t(sms) * 8;
  k<<<unsigned(ctas < most ? ctas : most), pisa::kCacheThreads, 0, st>>>(p);
  return check_launch(what);
}

// make_map with a box of box2 slices: tiles of several heads' tokens
pisa_status_t make_rows_map(CUtensorMap* m, const void* ptr, uint64_t d0, uint64_t d1, uint64_t d2, uint32_t box1,
                            uint32_t box2) {
  auto fn = encode_fn();
  if (!fn) return fail(PISA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  cuuint64_t dims[3] = {d0, d1, d2};
  cuuint64_t strides[2] = {d0 * 2, d0 * d1 * 2};
  cuuint32_t box[3] = {64, box1, box2};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(PISA_ERR_CUDA, "cuTensorMapEncodeTiled (rows) failed (%d)", int(r));
  return ok();
}

// codes of 8 bits [d2][d1][d0], box {d0, box1, 1}, rows contiguous in shared memory
pisa_status_t make_code_map(CUtensorMap* m, const void* ptr, uint64_t d0, uint64_t d1, uint64_t d2, uint32_t box1) {
  auto fn = encode_fn();
  if (!fn) return fail(PISA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  cuuint64_t dims[3] = {d0, d1, d2};
  cuuint64_t strides[2] = {d0, d0 * d1};
  cuuint32_t box[3] = {uint32_t(d0), box1, 1};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(PISA_ERR_CUDA, "cuTensorMapEncodeTiled (codes) failed (%d)", int(r));
  return ok();
}

// Pieces of two row tiles, and the runs that their tiles are cut into so that few rows over a long
// cache still fill the SMs. Time goes as waves of (tiles of a run + a piece's own cost, about two
// tiles; three with the partial sums of a cut one): the cut with the least is taken, of at least
// two tiles a run.
constexpr int kSms = 148;
void plan_attend(pisa::AttendTcParams* p, int64_t keys) {
  p->rt = pisa::RowTiles::of(p->Hq / p->Hkv);
  p->G = p->Hq / p->Hkv;
  p->part_pairs = int((int64_t(p->N) + 2 * p->rt.tokens - 1) / (2 * p->rt.tokens));
  p->pairs = p->rt.parts * p->part_pairs;
  const int64_t pieces = int64_t(p->B) * p->Hkv * p->pairs, tiles = (keys + 127) / 128;
  int64_t best = 1;
  double least = 1e300;
  for (int64_t s = 1; s <= kSms && (s == 1 || (s <= tiles / 2 && (s - 1) * pieces < 2 * kSms)); ++s) {
    const double waves = double((pieces * s + kSms - 1) / kSms);
    const double cost = waves * (double((tiles + s - 1) / s) + (s > 1 ? 3.0 : 2.0));
    if (cost < least * 0.97) {
      least = cost;
      best = s;
    }
  }
  p->splits = int(best);
  p->items = int(pieces * best);
}
size_t attend_workspace(const pisa::AttendTcParams& p, int d) {
  return p.splits > 1 ? size_t(p.splits) * p.B * p.Hq * p.N * (size_t(d) + 1) * 4 : 0;
}

// A kernel whose blocks start as the last ones of the kernel before it run (which lets them with
// griddepcontrol.launch_dependents); they set up and wait (griddepcontrol.wait) for it to end.
template <class... Args>
pisa_status_t launch_behind(void (*kernel)(Args...), unsigned grid, unsigned block, size_t smem, cudaStream_t st,
                            const char* name, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) return fail(PISA_ERR_CUDA, "%s launch: %s", name, cudaGetErrorString(e));
  return check_launch(name);
}

template <int D, int KV>
pisa_status_t launch_attend_tc(pisa::AttendTcParams p, const void* K, const void* V, int page, int num_pages,
                               void* workspace, cudaStream_t st) {
  using C = pisa::AttendTcCfg<D, KV>;
  const int ctas = p.items < kSms ? p.items : kSms;
  // twice the cycles that a pair of tiles takes, for every tile of the CTA's items
  const int64_t cap = KV == pisa::kKvPlain ? p.N : int64_t(p.pages.max_pages) * page;
  p.patience = int64_t((p.items + ctas - 1) / ctas) * (cap / 128 / p.splits + 2) * 8192;
  CUtensorMap mQ, mK, mV;
  PISA_TRY(make_rows_map(&mQ, p.Q, D, uint64_t(p.N), uint64_t(p.B) * p.Hq, uint32_t(p.rt.tokens), uint32_t(p.rt.heads)));
  if constexpr (KV == pisa::kKvPlain) {
    PISA_TRY(make_map(&mK, K, D, uint64_t(p.N), uint64_t(p.B) * p.Hkv, 128));
    PISA_TRY(make_map(&mV, V, D, uint64_t(p.N), uint64_t(p.B) * p.Hkv, 128));
    p.pages.K = K;
    p.pages.V = V;
  } else if constexpr (KV == pisa::kKvPaged) {
    PISA_TRY(make_map(&mK, K, D, uint64_t(page), uint64_t(num_pages) * p.Hkv, uint32_t(page)));
    PISA_TRY(make_map(&mV, V, D, uint64_t(page), uint64_t(num_pages) * p.Hkv, uint32_t(page)));
  } else {
    PISA_TRY(make_code_map(&mK, K, D, uint64_t(page), uint64_t(num_pages) * p.Hkv, uint32_t(page)));
    PISA_TRY(make_code_map(&mV, V, D, uint64_t(page), uint64_t(num_pages) * p.Hkv, uint32_t(page)));
  }
  const int64_t rows = int64_t(p.B) * p.Hq * p.N;
  const bool runs = KV != pisa::kKvPlain && p.splits > 1;
  if (runs) {
    p.part = static_cast<float*>(workspace);
    p.part_lse = p.part + size_t(p.splits) * rows * D;
  }
  auto k = pisa::attend_tc_kernel<D, KV>;
  PISA_TRY(set_smem(k, C::SMEM));
  k<<<unsigned(ctas), C::kThreads, C::SMEM, st>>>(mQ, mK, mV, p);
  PISA_TRY(check_launch("attend_tc_kernel"));
  if constexpr (KV != pisa::kKvPlain) {
    constexpr int per = pisa::kJoinThreads / (D / 4);  // rows of a block
    if (runs)
      PISA_TRY(launch_behind(pisa::attend_join_kernel<D>, unsigned((rows + per - 1) / per), pisa::kJoinThreads, 0, st,
                             "attend_join_kernel", p));
  }
  return ok();
}

// sizes and plan of a paged call (the longest sequence the table can hold, or the window's reach)
pisa::AttendTcParams paged_plan(const pisa_cache_t& c, const pisa_sequences_t& s, int32_t Hq, const pisa::Pages& g,
                                const pisa::Window& w, int64_t* keys) {
  pisa::AttendTcParams a{};
  a.pages = g;
  a.B = s.B;
  a.Hq = Hq;
  a.Hkv = c.Hkv;
  a.N = s.N;
  a.win = w;
  const int64_t cap = int64_t(s.max_pages) * c.page;
  const int64_t seen = int64_t(w.left) + w.right + s.N + w.sinks;
  *keys = seen < cap ? seen : cap;
  plan_attend(&a, *keys);
  return a;
}

// Up to 16 rows per key head: the token kernel. As many CTAs as the SMs hold at once, fewer if
// the cache cannot hold as many chunks.
bool few_rows(const pisa::AttendTcParams& a) { return int64_t(a.Hq / a.Hkv) * a.N <= pisa::kTokenRows; }
int token_ctas(const pisa::AttendTcParams& a, int64_t keys, int d, int type) {
  const int64_t chunk = pisa::kTokenWarps * pisa::token_keys(d);
  const int64_t most = int64_t(a.B) * a.Hkv * ((keys + chunk - 1) / chunk + 1);
  const bool wide = int64_t(a.Hq / a.Hkv) * a.N > 8, codes = type == PISA_CACHE_E4M3;
  const int fit = wide ? (codes ? pisa::token_ctas_per_sm<128, true, 2>() : pisa::token_ctas_per_sm<128, false, 2>())
                       : (codes ? pisa::token_ctas_per_sm<128, true, 1>() : pisa::token_ctas_per_sm<128, false, 1>());
  return int(most < int64_t(fit) * kSms ? most : int64_t(fit) * kSms);
}
size_t token_workspace(int ctas, int d) { return size_t(2) * ctas * pisa::kTokenRows * (size_t(d) + 1) * 4; }

template <int D, bool E4M3>
pisa_status_t launch_token(const pisa::AttendTcParams& a, int ctas, void* workspace, cudaStream_t st) {
  pisa::AttendTokenParams p{a.Q, a.O, a.lse, static_cast<float*>(workspace), nullptr, a.pages, a.B, a.Hq, a.Hkv, a.N,
                            ctas, a.win, a.scale};
  p.part_lse = p.part + size_t(2) * ctas * pisa::kTokenRows * D;
  const int64_t rows = int64_t(a.Hq / a.Hkv) * a.N;
  auto k = rows > 8 ? pisa::attend_token_kernel<D, E4M3, 2> : pisa::attend_token_kernel<D, E4M3, 1>;
  k<<<unsigned(ctas), 32 * pisa::kTokenWarps, 0, st>>>(p);
  PISA_TRY(check_launch("attend_token_kernel"));
  PISA_TRY(launch_behind(pisa::attend_token_join_kernel<D>, unsigned(a.B * a.Hkv * rows), 32 * pisa::kTokenWarps, 0, st,
                         "attend_token_join_kernel", p));
  return ok();
}

// How the key tiles of the gradient are cut into runs of query tiles: as if two CTAs per SM shared
// all of them evenly, so that a tile which every row sees (the first tokens, or a causal sequence's
// first keys) is cut and a window's are not. (Runs of the window's own length, with more partial sums,
// measured 2% slower: 1306 against 1277 us for the step on 16384 tokens.)
struct GradPlan {
  int run, runs, slots;
  size_t delta_bytes, bytes;
};
GradPlan plan_grad(const pisa_window_shape_t& s, const pisa::Window& w) {
  const int kts = (s.N + 127) / 128, G = s.Hq / s.Hkv;
  const int64_t heads = int64_t(s.B) * s.Hkv;
  int64_t total = 0;
  for (int kt = 0; kt < kts; ++kt) total += int64_t(G) * pisa::QueryRange(w, kt, s.N).count;
  const int64_t run = (total * heads + 2 * kSms - 1) / (2 * kSms);
  GradPlan g{};
  g.run = int(run < 16 ? 16 : (run > INT32_MAX ? INT32_MAX : run));
  for (int kt = 0; kt < kts; ++kt) {
    const int r = pisa::query_runs(G * pisa::QueryRange(w, kt, s.N).count, g.run);
    g.runs += r;
    if (r > 1) g.slots += r;
  }
  g.delta_bytes = (size_t(s.B) * s.Hq * s.N * 4 + 255) / 256 * 256;
  g.bytes = g.delta_bytes + size_t(heads) * g.slots * 2 * 128 * s.d * 4;
  return g;
}

template <int D>
pisa_status_t launch_grad(pisa::AttendGradParams p, const GradPlan& g, const void* K, const void* V, cudaStream_t st) {
  const uint64_t heads = uint64_t(p.B) * p.Hkv, q_heads = uint64_t(p.B) * p.Hq, N = uint64_t(p.N);
  p.rt = pisa::RowTiles::of(p.Hq / p.Hkv);
  CUtensorMap mK, mV, mQ, mG, rQ, rG, rO;
  PISA_TRY(make_rows_map(&rQ, p.Q, D, N, q_heads, uint32_t(p.rt.tokens), uint32_t(p.rt.heads)));
  PISA_TRY(make_rows_map(&rG, p.dO, D, N, q_heads, uint32_t(p.rt.tokens), uint32_t(p.rt.heads)));
  PISA_TRY(make_rows_map(&rO, p.O, D, N, q_heads, uint32_t(p.rt.tokens), uint32_t(p.rt.heads)));
  PISA_TRY(make_map(&mK, K, D, N, heads, 128));
  PISA_TRY(make_map(&mV, V, D, N, heads, 128));
  PISA_TRY(make_map(&mQ, p.Q, D, N, q_heads, 64));
  PISA_TRY(make_map(&mG, p.dO, D, N, q_heads, 64));
  auto kq = pisa::attend_dq_kernel<D>;
  auto kk = pisa::attend_dkv_kernel<D>;
  using Cq = pisa::AttendDqCfg<D>;
  using Ck = pisa::AttendDkvCfg<D>;
  PISA_TRY(set_smem(kq, Cq::SMEM));
  PISA_TRY(set_smem(kk, Ck::SMEM));
  const unsigned row_tiles = unsigned(p.rt.parts) * unsigned((p.N + p.rt.tokens - 1) / p.rt.tokens);
  kq<<<row_tiles * unsigned(heads), Cq::kThreads, Cq::SMEM, st>>>(rQ, rG, rO, mK, mV, p);
  PISA_TRY(check_launch("attend_dq_kernel"));
  PISA_TRY(launch_behind(kk, unsigned(g.runs) * unsigned(heads), Ck::kThreads, Ck::SMEM, st, "attend_dkv_kernel", mK, mV, mQ,
                         mG, p));
  if (g.slots > 0)
    PISA_TRY(launch_behind(pisa::attend_dkv_join_kernel<D>, unsigned((N + 127) / 128 * heads) * pisa::kJoinSlices, 256, 0, st,
                           "attend_dkv_join_kernel", p));
  return ok();
}

}  // namespace

extern "C" {

pisa_status_t pisa_window_attention(const void* Q, const void* K, const void* V, pisa_window_shape_t shape,
                                    pisa_window_t window, float scale, void* O, float* lse, void* stream) {
  bool empty = false;
  PISA_TRY(check_heads(shape.B, shape.Hq, shape.Hkv, shape.N, shape.d, &empty));
  pisa::AttendTcParams a{};
  PISA_TRY(check_window(window, &a.win));
  PISA_TRY(check_scale(scale));
  if (empty) return ok();
  PISA_TRY(check_ptr(Q, "Q"));
  PISA_TRY(check_ptr(K, "K"));
  PISA_TRY(check_ptr(V, "V"));
  PISA_TRY(check_ptr(O, "O"));
  if (lse != nullptr) PISA_TRY(check_aligned(lse, "lse", 4));
  int sms = 0;
  PISA_TRY(check_device(&sms));
  a.Q = static_cast<const bf16*>(Q);
  a.O = static_cast<bf16*>(O);
  a.lse = lse;
  a.B = shape.B;
  a.Hq = shape.Hq;
  a.Hkv = shape.Hkv;
  a.N = shape.N;
  a.scale = scale;
  plan_attend(&a, 0);  // no runs: the call has no workspace for their sums, and few heads leave SMs idle
  auto st = static_cast<cudaStream_t>(stream);
  return shape.d == 128 ? launch_attend_tc<128, pisa::kKvPlain>(a, K, V, 0, 0, nullptr, st)
                        : launch_attend_tc<64, pisa::kKvPlain>(a, K, V, 0, 0, nullptr, st);
}

pisa_status_t pisa_window_attention_backward_workspace(pisa_window_shape_t shape, pisa_window_t window,
                                                       size_t* bytes) {
  if (bytes == nullptr) return fail(PISA_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = 0;
  bool empty = false;
  PISA_TRY(check_heads(shape.B, shape.Hq, shape.Hkv, shape.N, shape.d, &empty));
  pisa::Window w;
  PISA_TRY(check_window(window, &w));
  if (empty) return ok();
  *bytes = plan_grad(shape, w).bytes;
  return ok();
}

pisa_status_t pisa_window_attention_backward(const void* dO, const void* Q, const void* K, const void* V,
                                             const void* O, const float* lse, pisa_window_shape_t shape,
                                             pisa_window_t window, float scale, void* dQ, void* dK, void* dV,
                                             void* workspace, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  PISA_TRY(pisa_window_attention_backward_workspace(shape, window, &need));
  PISA_TRY(check_scale(scale));
  if (need == 0) return ok();  // empty problem: nothing touched
  pisa::AttendGradParams p{};
  PISA_TRY(check_window(window, &p.win));
  const void* bufs[8] = {dO, Q, K, V, O, dQ, dK, dV};
  const char* names[8] = {"dO", "Q", "K", "V", "O", "dQ", "dK", "dV"};
  for (int i = 0; i < 8; ++i) PISA_TRY(check_ptr(bufs[i], names[i]));
  PISA_TRY(check_aligned(lse, "lse", 4));
  PISA_TRY(check_workspace(workspace, workspace_bytes, need));
  int sms = 0;
  PISA_TRY(check_device(&sms));
  p.Q = static_cast<const bf16*>(Q);
  p.O = static_cast<const bf16*>(O);
  p.lse = lse;
  p.dO = static_cast<const bf16*>(dO);
  p.dQ = static_cast<bf16*>(dQ);
  p.dK = static_cast<bf16*>(dK);
  p.dV = static_cast<bf16*>(dV);
  p.delta = static_cast<float*>(workspace);
  p.B = shape.B;
  p.Hq = shape.Hq;
  p.Hkv = shape.Hkv;
  p.N = shape.N;
  p.scale = scale;
  const GradPlan g = plan_grad(shape, p.win);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + g.delta_bytes);
  p.run = g.run;
  p.runs = g.runs;
  p.slots = g.slots;
  auto st = static_cast<cudaStream_t>(stream);
  return shape.d == 128 ? launch_grad<128>(p, g, K, V, st) : launch_grad<64>(p, g, K, V, st);
}

pisa_status_t pisa_cache_write(const void* K, const void* V, pisa_cache_t cache, pisa_sequences_t seqs,
                               void* stream) {
  bool empty = false;
  pisa::CacheParams p{};
  PISA_TRY(check_cache(cache, seqs, cache.Hkv, &empty, &p.pages));
  if (empty) return ok();
  PISA_TRY(check_ptr(K, "K"));
  PISA_TRY(check_ptr(V, "V"));
  int sms = 0;
  PISA_TRY(check_device(&sms));
  p.cK = cache.K;
  p.cV = cache.V;
  p.ks = cache.k_scale;
  p.vs = cache.v_scale;
  p.K = static_cast<const bf16*>(K);
  p.V = static_cast<const bf16*>(V);
  p.Hkv = cache.Hkv;
  p.N = seqs.N;
  p.rows = int64_t(seqs.B) * cache.Hkv * seqs.N;
  auto st = static_cast<cudaStream_t>(stream);
  const bool q = cache.type == PISA_CACHE_E4M3;
  auto k = cache.d == 128 ? (q ? pisa::cache_write_kernel<128, true> : pisa::cache_write_kernel<128, false>)
                          : (q ? pisa::cache_write_kernel<64, true> : pisa::cache_write_kernel<64, false>);
  return launch_cache(k, p, cache.d, q ? 32 : 8, sms, st, "cache_write_kernel");
}

pisa_status_t pisa_cache_read(pisa_cache_t cache, pisa_sequences_t seqs, void* K, void* V, void* stream) {
  bool empty = false;
  pisa::CacheParams p{};
  seqs.q_lens = nullptr;
  PISA_TRY(check_cache(cache, seqs, cache.Hkv, &empty, &p.pages));
  if (empty) return ok();
  PISA_TRY(check_ptr(K, "K"));
  PISA_TRY(check_ptr(V, "V"));
  int sms = 0;
  PISA_TRY(check_device(&sms));
  p.oK = static_cast<bf16*>(K);
  p.oV = static_cast<bf16*>(V);
  p.Hkv = cache.Hkv;
  p.N = seqs.N;
  p.rows = int64_t(seqs.B) * cache.Hkv * seqs.N;
  auto st = static_cast<cudaStream_t>(stream);
  const bool q = cache.type == PISA_CACHE_E4M3;
  auto k = cache.d == 128 ? (q ? pisa::cache_read_kernel<128, true> : pisa::cache_read_kernel<128, false>)
                          : (q ? pisa::cache_read_kernel<64, true> : pisa::cache_read_kernel<64, false>);
  return launch_cache(k, p, cache.d, q ? 16 : 8, sms, st, "cache_read_kernel");
}

pisa_status_t pisa_paged_attention_workspace(pisa_cache_t cache, pisa_sequences_t seqs, int32_t Hq,
                                             pisa_window_t window, size_t* bytes) {
  if (bytes == nullptr) return fail(PISA_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = 0;
  bool empty = false;
  pisa::Pages g{};
  PISA_TRY(check_cache(cache, seqs, Hq, &empty, &g));
  pisa::Window w;
  PISA_TRY(check_window(window, &w));
  if (empty) return ok();
  int64_t keys = 0;
  const pisa::AttendTcParams a = paged_plan(cache, seqs, Hq, g, w, &keys);
  *bytes = few_rows(a) ? token_workspace(token_ctas(a, keys, cache.d, cache.type), cache.d)
                       : attend_workspace(a, cache.d);
  return ok();
}

pisa_status_t pisa_paged_attention(const void* Q, pisa_cache_t cache, pisa_sequences_t seqs, int32_t Hq,
                                   pisa_window_t window, float scale, void* O, float* lse, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  bool empty = false;
  pisa::Pages g{};
  pisa::Window w;
  PISA_TRY(check_cache(cache, seqs, Hq, &empty, &g));
  PISA_TRY(check_window(window, &w));
  PISA_TRY(check_scale(scale));
  if (empty) return ok();
  PISA_TRY(check_ptr(Q, "Q"));
  PISA_TRY(check_ptr(O, "O"));
  if (lse != nullptr) PISA_TRY(check_aligned(lse, "lse", 4));
  size_t need = 0;
  PISA_TRY(pisa_paged_attention_workspace(cache, seqs, Hq, window, &need));
  PISA_TRY(check_workspace(workspace, workspace_bytes, need));
  int sms = 0;
  PISA_TRY(check_device(&sms));
  int64_t keys = 0;
  pisa::AttendTcParams a = paged_plan(cache, seqs, Hq, g, w, &keys);
  a.Q = static_cast<const bf16*>(Q);
  a.O = static_cast<bf16*>(O);
  a.lse = lse;
  a.scale = scale;
  auto st = static_cast<cudaStream_t>(stream);
  const bool codes = cache.type == PISA_CACHE_E4M3;
  if (few_rows(a)) {
    const int ctas = token_ctas(a, keys, cache.d, cache.type);
    if (codes)
      return cache.d == 128 ? launch_token<128, true>(a, ctas, workspace, st) : launch_token<64, true>(a, ctas, workspace, st);
    return cache.d == 128 ? launch_token<128, false>(a, ctas, workspace, st) : launch_token<64, false>(a, ctas, workspace, st);
  }
  const auto run = [&](auto k) { return k(a, cache.K, cache.V, cache.page, cache.num_pages, workspace, st); };
  if (codes)
    return cache.d == 128 ? run(launch_attend_tc<128, pisa::kKvPagedE4m3>) : run(launch_attend_tc<64, pisa::kKvPagedE4m3>);
  return cache.d == 128 ? run(launch_attend_tc<128, pisa::kKvPaged>) : run(launch_attend_tc<64, pisa::kKvPaged>);
}

}  // extern "C"
