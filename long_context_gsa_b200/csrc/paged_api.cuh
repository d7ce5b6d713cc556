// paged_api.cuh -- the entry points of the paged raw-token cache (see
// include/gsa.h): argument checks, split sizing and launches.  Included by
// gsa_api.cu behind its own entry points, whose helpers it uses.
#pragma once

#include <atomic>

namespace gsa {
namespace {

gsa_status check_paged(const gsa_desc *d, const gsa_pdesc *p) {
  GSA_TRY(check_desc(d));
  if (!p) return GSA_ERR_INVALID_ARG;
  if (p->cache_dtype < GSA_F32 || p->cache_dtype > GSA_E4M3) return GSA_ERR_INVALID_ARG;
  if (p->page < 1 || p->page % d->chunk || p->n_pages < 1 || p->max_pages < 1) return GSA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(p->max_pages) * p->page < d->t_max) return GSA_ERR_INVALID_ARG;
  if (p->page > (1 << 28) || d->batch > kPgMaxBatch || d->hq > 65535) return GSA_ERR_UNSUPPORTED;
  // rows of the pool are counted in 32 bits
  if (static_cast<int64_t>(p->n_pages) * p->page >= (int64_t(1) << 32) / d->hkv) return GSA_ERR_UNSUPPORTED;
  return GSA_OK;
}

// The readers: 8-bit codes only.
gsa_status check_paged_read(const gsa_desc *d, const gsa_pdesc *p, const void *k, const void *v, const float *ks,
                            const float *vs, const int32_t *table) {
  GSA_TRY(check_paged(d, p));
  if (p->cache_dtype != GSA_I8 && p->cache_dtype != GSA_E4M3) return GSA_ERR_UNSUPPORTED;
  for (const void *x : {k, v, static_cast<const void *>(ks), static_cast<const void *>(vs),
                        static_cast<const void *>(table)})
    GSA_TRY(need_ptr(x));
  return GSA_OK;
}

PagedKV paged_kv(const gsa_desc *d, const gsa_pdesc *p, const void *k, const void *v, const float *ks, const float *vs,
                 const int32_t *table) {
  PagedKV kv;
  kv.k = static_cast<const uint8_t *>(k);
  kv.v = static_cast<const uint8_t *>(v);
  kv.ks = ks;
  kv.vs = vs;
  kv.table = table;
  kv.n_pages = p->n_pages;
  kv.max_pages = p->max_pages;
  kv.hkv = d->hkv;
  kv.blocks = p->page / d->chunk;
  kv.page.init(p->page);
  kv.chunk.init(d->chunk);
  return kv;
}

// fn(D, format, fp32 queries) as compile-time constants.
template <typename Fn>
gsa_status paged_variant(const gsa_desc *d, const gsa_pdesc *p, Fn fn) {
  using I8 = std::integral_constant<int, kFmtI8>;
  using E4 = std::integral_constant<int, kFmtE4M3>;
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  auto with = [&](auto dim, auto fmt) {
    return d->dtype == GSA_F32 ? fn(dim, fmt, std::true_type()) : fn(dim, fmt, std::false_type());
  };
  if (d->d == 64) return p->cache_dtype == GSA_I8 ? with(D64(), I8()) : with(D64(), E4());
  return p->cache_dtype == GSA_I8 ? with(D128(), I8()) : with(D128(), E4());
}

// CTAs of one kernel that fit on the whole GPU, remembered for each device and
// the amount of shared memory asked for last (the queries cost microseconds, as
// much as a small call's kernel); 0 on an error.  The kernel is allowed all the
// shared memory there is, once: launches from several threads with different
// amounts must not lower one another's limit.
struct SlotCache {
  static constexpr int kDevices = 16;
  std::atomic<uint64_t> known[kDevices] = {};  // smem << 32 | CTAs
  template <typename Kern>
  int get(Kern kern, int threads, size_t smem) {
    int dev = -1;
    const bool keep = cudaGetDevice(&dev) == cudaSuccess && dev >= 0 && dev < kDevices;
    if (keep) {
      const uint64_t v = known[dev].load(std::memory_order_relaxed);
      if (v && (v >> 32) == smem) return static_cast<int>(v & 0xffffffffu);
    }
    cudaFuncAttributes fa;
    int optin = 0, per_sm = 0;
    if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess ||
        cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess ||
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             optin - static_cast<int>(fa.sharedSizeBytes)) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem) != cudaSuccess || per_sm < 1) {
      cudaGetLastError();
      return 0;
    }
    const int n = per_sm * sm_count();
    if (keep) known[dev].store(static_cast<uint64_t>(smem) << 32 | static_cast<uint32_t>(n), std::memory_order_relaxed);
    return n;
  }
};

template <int D, int FMT, bool QF32, int NT>
gsa_status launch_paged_attend(const PagedAttendArgs &pa, void *stream) {
  const size_t smem = paged_attend_smem<D, FMT, QF32, NT>() + (2 * static_cast<size_t>(pa.B) + 1) * 4;
  const auto kern = k_paged_attend<D, FMT, QF32, NT>;
  static SlotCache cache;
  const int grid = std::min(kPgMaxCtas, cache.get(kern, kPgThreads, smem));
  if (grid < 1) return GSA_ERR_CUDA;
  GSA_TRY(launch_prepared(kern, dim3(grid), dim3(kPgThreads), smem, stream, pa));
  // no segment can have been cut when the longest is short
  if (pa.t_max <= static_cast<int>(kPgWhole) * kPgStep) return GSA_OK;
  const size_t weights = static_cast<size_t>(grid) * 8 * 4;
  // Four warps a row where a segment has many records, 12 or more if all are of length t_max; one where it has few and
  // the join is short: 1 x 32K rows of d = 64 (74 records) 21.7 and 23.6 us, 1 x 128K of d = 128 (111) 47.4 and 56.9,
  // 4 x 32K (18) 34.3 and 34.8; 16 x 32K of d = 128 (7) 113.0 and 112.1, of d = 64 (5) 98.9 and 98.1, 32 x 8K of
  // d = 128 (3) 68.3 and 67.0, 16 x 2K of d = 64 (5) 18.6 and 17.7.
  const int64_t segments = static_cast<int64_t>(pa.B) * pa.kv.hkv * pa.rg;
  const int longest = (cdiv(pa.t_max, kPgStep) + static_cast<int>(kPgHead)) / pa.min_steps;
  if (std::min<int64_t>(grid / segments, longest) >= 12)
    return launch(k_paged_join<D, NT, 4>, dim3(grid, 4 * NT), dim3(256), weights, stream, pa);
  return launch(k_paged_join<D, NT, 1>, dim3(grid, NT), dim3(256), weights, stream, pa);
}

gsa_status run_paged_unfold(const gsa_desc *d, const gsa_pdesc *p, const void *q, const void *k, const void *v,
                            const float *ks, const float *vs, const int32_t *table, const void *gist_v,
                            const int32_t *n_gists, const int32_t *own_len, const int32_t *sel_idx,
                            const float *sel_score, const float *prior, int n_prior, void *out, float *lse,
                            const Layout &L, void *ws, void *stream, bool armed, uint32_t *ready = nullptr) {
  PagedUnfoldArgs pa;
  std::memset(static_cast<void *>(&pa), 0, sizeof(pa));
  UnfoldArgs &ua = pa.u;
  ua.q = q;
  ua.gist_v = gist_v;
  ua.n_gists = n_gists;
  ua.own_len = own_len;
  ua.sel_idx = sel_idx;
  ua.sel_score = sel_score;
  ua.k = d->topk;
  ua.chunk = d->chunk;
  ua.t_max = d->t_max;
  ua.n_max = d->n_max;
  ua.hq = d->hq;
  ua.hkv = d->hkv;
  ua.group = d->hq / d->hkv;
  ua.exclude = d->exclude_unselected;
  ua.scale_log2 = resolve_scale(d) * kLog2e;
  ua.part = reinterpret_cast<float *>(at(ws, L.part_u));
  ua.prior = prior;
  ua.n_prior = prior ? n_prior : 0;
  ua.counters = reinterpret_cast<uint32_t *>(at(ws, L.counters));
  ua.ready.w = ready;
  ua.ready.rows = d->batch * d->hq;
  ua.status = reinterpret_cast<uint32_t *>(at(ws, L.status));
  ua.out = out;
  ua.out_bf16 = d->out_dtype == GSA_BF16;
  ua.lse = lse;
  pa.kv = paged_kv(d, p, k, v, ks, vs, table);
  return paged_variant(d, p, [&](auto dim, auto fmt, auto qf32) {
    constexpr int D = decltype(dim)::value, F = decltype(fmt)::value;
    constexpr bool Q = decltype(qf32)::value;
    const auto kern = k_paged_unfold<D, F, Q>;
    // residency with the largest list share (one split), then the share of the chosen split count; a split is
    // not made smaller than one 32-row tile a warp
    const int k1 = std::max(1, ua.k);
    static SlotCache cache;
    const int slots = cache.get(kern, kUnfoldThreads, paged_unfold_smem<D, F, Q>(k1));
    if (slots < 1) return GSA_ERR_CUDA;
    const int most = std::max(1, static_cast<int>(static_cast<int64_t>(k1) * d->chunk / (32 * kPuWarps)));
    ua.n_split = one_wave_splits(d->batch * d->hq, slots, std::min(std::min(kUnfoldSplitMax, k1), most));
    // The rows' counters must be zero.  In the fused step the scoring or the selection has re-armed them; here a
    // kernel does (0.5 us of 17; a memset, which no kernel starts ahead of, 4).
    if (ua.n_split > 1 && !armed)
      GSA_TRY(launch_prepared(k_paged_arm, dim3(cdiv(ua.ready.rows, 256)), dim3(256), 0, stream, ua.counters,
                              ua.ready.rows));
    return launch_prepared(kern, dim3(ua.n_split, d->hq, d->batch), dim3(kUnfoldThreads),
                           paged_unfold_smem<D, F, Q>(cdiv(k1, ua.n_split)), stream, pa);
  });
}

template <int D, typename T, int FMT, bool INTER>
gsa_status launch_append(const AppendArgs &aa, void *stream) {
  // an upper bound of the touched blocks: a sequence's first and last one may be part-filled
  const int chunk = static_cast<int>(aa.chunk.d);
  const int64_t most = std::min<int64_t>(aa.n_tok, aa.n_tok / chunk + 2 * static_cast<int64_t>(aa.B));
  const size_t smem = (8 + static_cast<size_t>(chunk) * (aa.rot / 2)) * 8 + (static_cast<size_t>(aa.B) + 1) * 4;
  const auto kern = k_paged_append<D, T, FMT, INTER>;
  static SlotCache cache;
  const int slots = cache.get(kern, kApThreads, smem);
  if (slots < 1) return GSA_ERR_CUDA;
  const int x = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(most, slots)));
  // few blocks: several CTAs share the heads of each, one task a warp
  const int rows = static_cast<int>((aa.n_tok + most - 1) / most);
  const int tasks = 2 * aa.hkv + (aa.q ? rows * cdiv(aa.hq, kQPass * 32 / (D / 16)) : 0);
  const int y = clampi(slots / x, 1, cdiv(tasks, kApWarps));
  return launch_prepared(kern, dim3(x, y), dim3(kApThreads), smem, stream, aa);
}

}  // namespace
}  // namespace gsa

extern "C" {

gsa_status gsa_paged_append(const gsa_desc *desc, const gsa_pdesc *pdesc, const gsa_append_desc *adesc,
                            const void *q_new, const void *k_new, const void *v_new, const int32_t *cu_tok,
                            const int32_t *pos, const float *inv_freq, const int32_t *page_table,
                            const int32_t *n_gists, int32_t *own_len, void *k_pages, void *v_pages, float *k_scale,
                            float *v_scale, void *q_out, void *ws, size_t ws_bytes, void *stream) {
  GSA_TRY(check_paged(desc, pdesc));
  if (!adesc) return GSA_ERR_INVALID_ARG;
  const bool coded = pdesc->cache_dtype == GSA_I8 || pdesc->cache_dtype == GSA_E4M3;
  if (!coded && pdesc->cache_dtype != desc->dtype) return GSA_ERR_UNSUPPORTED;
  if (adesc->n_tok < 0 || adesc->rot_dim < 0 || adesc->rot_dim > desc->d) return GSA_ERR_INVALID_ARG;
  if (adesc->rot_dim % 16) return GSA_ERR_UNSUPPORTED;
  if ((adesc->interleaved | 1) != 1 || (adesc->advance | 1) != 1) return GSA_ERR_INVALID_ARG;
  if (!cu_tok && adesc->n_tok % desc->batch) return GSA_ERR_INVALID_ARG;
  const int64_t unit = 16 / static_cast<int64_t>(elem_size(desc->dtype));
  const int64_t q_row = static_cast<int64_t>(desc->hq) * desc->d, kv_row = static_cast<int64_t>(desc->hkv) * desc->d;
  const int64_t qs = adesc->q_stride ? adesc->q_stride : q_row;
  const int64_t ks = adesc->k_stride ? adesc->k_stride : kv_row;
  const int64_t vs = adesc->v_stride ? adesc->v_stride : kv_row;
  if (qs < q_row || ks < kv_row || vs < kv_row || qs % unit || ks % unit || vs % unit) return GSA_ERR_INVALID_ARG;
  for (const void *x : {static_cast<const void *>(page_table), static_cast<const void *>(own_len),
                        static_cast<const void *>(k_pages), static_cast<const void *>(v_pages),
                        static_cast<const void *>(ws)})
    GSA_TRY(need_ptr(x));
  if (adesc->n_tok > 0) {
    GSA_TRY(need_ptr(k_new));
    GSA_TRY(need_ptr(v_new));
  }
  for (const void *x : {q_new, static_cast<const void *>(cu_tok), static_cast<const void *>(pos),
                        static_cast<const void *>(n_gists)})
    GSA_TRY(opt_ptr(x));
  if (adesc->rot_dim) GSA_TRY(need_ptr(inv_freq));
  if (coded) {
    GSA_TRY(need_ptr(k_scale));
    GSA_TRY(need_ptr(v_scale));
  }
  if (q_new) {
    GSA_TRY(need_ptr(q_out));
    if (q_out == q_new) return GSA_ERR_INVALID_ARG;  // queries are read as data that nobody writes meanwhile
  }
  const Layout L = layout(desc, GSA_OP_PAGED, nullptr);
  if (ws_bytes < L.total) return GSA_ERR_WORKSPACE;
  if (adesc->n_tok == 0) return GSA_OK;
  AppendArgs aa;
  aa.q = q_new;
  aa.k = k_new;
  aa.v = v_new;
  aa.cu = cu_tok;
  aa.pos = pos;
  aa.inv_freq = inv_freq;
  aa.table = page_table;
  aa.n_gists = n_gists;
  aa.own_len = own_len;
  aa.kp = k_pages;
  aa.vp = v_pages;
  aa.ks = k_scale;
  aa.vs = v_scale;
  aa.q_out = q_out;
  aa.q_stride = static_cast<int32_t>(qs);
  aa.k_stride = static_cast<int32_t>(ks);
  aa.v_stride = static_cast<int32_t>(vs);
  aa.n_tok = adesc->n_tok;
  aa.B = desc->batch;
  aa.hq = desc->hq;
  aa.hkv = desc->hkv;
  aa.n_max = desc->n_max;
  aa.t_max = desc->t_max;
  aa.n_pages = pdesc->n_pages;
  aa.max_pages = pdesc->max_pages;
  aa.blocks = pdesc->page / desc->chunk;
  aa.rot = adesc->rot_dim;
  aa.advance = adesc->advance;
  aa.page.init(pdesc->page);
  aa.chunk.init(desc->chunk);
  aa.counter = reinterpret_cast<uint32_t *>(at(ws, L.pg_append));
  aa.status = reinterpret_cast<uint32_t *>(at(ws, L.status));
  auto go = [&](auto type, auto inter) {
    using T = decltype(type);
    constexpr bool I = decltype(inter)::value;
    const bool d64 = desc->d == 64;
    if (pdesc->cache_dtype == GSA_I8)
      return d64 ? launch_append<64, T, kFmtI8, I>(aa, stream) : launch_append<128, T, kFmtI8, I>(aa, stream);
    if (pdesc->cache_dtype == GSA_E4M3)
      return d64 ? launch_append<64, T, kFmtE4M3, I>(aa, stream) : launch_append<128, T, kFmtE4M3, I>(aa, stream);
    return d64 ? launch_append<64, T, kFmtPlain, I>(aa, stream) : launch_append<128, T, kFmtPlain, I>(aa, stream);
  };
  if (desc->dtype == GSA_BF16)
    return adesc->interleaved ? go(__nv_bfloat16(), std::true_type()) : go(__nv_bfloat16(), std::false_type());
  return adesc->interleaved ? go(0.f, std::true_type()) : go(0.f, std::false_type());
}

gsa_status gsa_paged_attend(const gsa_desc *desc, const gsa_pdesc *pdesc, int32_t n_q, const void *q,
                            const void *k_pages, const void *v_pages, const float *k_scale, const float *v_scale,
                            const int32_t *page_table, const int32_t *n_gists, const int32_t *own_len, void *out,
                            float *lse, void *ws, size_t ws_bytes, void *stream) {
  GSA_TRY(check_paged_read(desc, pdesc, k_pages, v_pages, k_scale, v_scale, page_table));
  if (n_q < 1) return GSA_ERR_INVALID_ARG;
  if (n_q > kPgMaxQueries) return GSA_ERR_UNSUPPORTED;
  GSA_TRY(need_ptr(q));
  GSA_TRY(opt_ptr(n_gists));
  GSA_TRY(need_ptr(own_len));
  GSA_TRY(need_ptr(out));
  GSA_TRY(opt_ptr(lse));
  GSA_TRY(need_ptr(ws));
  const Layout L = layout(desc, GSA_OP_PAGED, nullptr);
  if (ws_bytes < L.total) return GSA_ERR_WORKSPACE;
  const int rows = n_q * (desc->hq / desc->hkv);
  // 8 query rows a segment, or 16 when there are more
  const bool wide = rows > 8;
  const int rg = cdiv(rows, wide ? 16 : 8);
  if (static_cast<int64_t>(desc->batch) * desc->hkv * rg >=
      (int64_t(1) << 31) / (cdiv(desc->t_max, kPgStep) + static_cast<int>(kPgHead)))
    return GSA_ERR_UNSUPPORTED;  // steps are counted in 32 bits
  PagedAttendArgs pa;
  pa.kv = paged_kv(desc, pdesc, k_pages, v_pages, k_scale, v_scale, page_table);
  pa.q = q;
  pa.n_gists = n_gists;
  pa.own_len = own_len;
  pa.B = desc->batch;
  pa.n_q = n_q;
  pa.hq = desc->hq;
  pa.group = desc->hq / desc->hkv;
  pa.rg = rg;
  pa.chunk = desc->chunk;
  pa.n_max = desc->n_max;
  pa.t_max = desc->t_max;
  // A CTA takes two steps at least: one sequence of 2000 rows takes 8.7 us with
  // 1, 9.2 with 2 and 10.6 with 4; 32 of up to 700 rows 17.5, 16.0 and 17.3.
  pa.min_steps = 2;
  pa.scale_log2 = resolve_scale(desc) * kLog2e;
  pa.part = reinterpret_cast<float *>(at(ws, L.pg_part));
  pa.joins = reinterpret_cast<int4 *>(at(ws, L.pg_joins));
  pa.status = reinterpret_cast<uint32_t *>(at(ws, L.status));
  pa.out = out;
  pa.out_bf16 = desc->out_dtype == GSA_BF16;
  pa.lse = lse;
  return paged_variant(desc, pdesc, [&](auto dim, auto fmt, auto qf32) {
    constexpr int D = decltype(dim)::value, F = decltype(fmt)::value;
    constexpr bool Q = decltype(qf32)::value;
    return wide ? launch_paged_attend<D, F, Q, 2>(pa, stream) : launch_paged_attend<D, F, Q, 1>(pa, stream);
  });
}

gsa_status gsa_paged_unfold(const gsa_desc *desc, const gsa_pdesc *pdesc, const void *q, const void *k_pages,
                            const void *v_pages, const float *k_scale, const float *v_scale,
                            const int32_t *page_table, const void *gist_v, const int32_t *n_gists,
                            const int32_t *own_len, const int32_t *sel_idx, const float *sel_score, int32_t prior,
                            void *out, float *lse, void *ws, size_t ws_bytes, void *stream) {
  GSA_TRY(check_paged_read(desc, pdesc, k_pages, v_pages, k_scale, v_scale, page_table));
  GSA_TRY(need_ptr(q));
  GSA_TRY(need_ptr(n_gists));
  GSA_TRY(need_ptr(own_len));
  GSA_TRY(need_ptr(out));
  GSA_TRY(opt_ptr(lse));
  GSA_TRY(need_ptr(ws));
  if (desc->topk > 0) GSA_TRY(need_ptr(sel_idx));
  if (desc->exclude_unselected && desc->topk > 0) {
    GSA_TRY(need_ptr(gist_v));
    GSA_TRY(need_ptr(sel_score));
  }
  if (prior != GSA_PRIOR_NONE && prior != GSA_PRIOR_GISTS && prior != GSA_PRIOR_HGSA && prior != GSA_PRIOR_HGSA2)
    return GSA_ERR_INVALID_ARG;
  if (prior == GSA_PRIOR_NONE && !desc->exclude_unselected) return GSA_ERR_INVALID_ARG;
  const Layout L = layout(desc, GSA_OP_DECODE, nullptr);  // the H-GSA and paged layouts extend this one
  if (ws_bytes < L.total) return GSA_ERR_WORKSPACE;
  const float *pr = nullptr;
  int n_prior = 0;
  if (prior != GSA_PRIOR_NONE && !desc->exclude_unselected) {
    pr = reinterpret_cast<const float *>(at(ws, L.part_g));
    n_prior = prior == GSA_PRIOR_GISTS ? gist_prior_count(desc)
                                       : (prior == GSA_PRIOR_HGSA ? 1 : 2) * hgsa_splits(desc);
  }
  return run_paged_unfold(desc, pdesc, q, k_pages, v_pages, k_scale, v_scale, page_table, gist_v, n_gists, own_len,
                          sel_idx, sel_score, pr, n_prior, out, lse, L, ws, stream, false);
}

gsa_status gsa_paged_decode(const gsa_desc *desc, const gsa_pdesc *pdesc, const void *q, const void *gist_k,
                            const void *gist_v, const void *k_pages, const void *v_pages, const float *k_scale,
                            const float *v_scale, const int32_t *page_table, const int32_t *n_gists,
                            const int32_t *own_len, void *out, float *lse, int32_t *sel_idx, float *sel_score,
                            void *ws, size_t ws_bytes, void *stream) {
  GSA_TRY(check_paged_read(desc, pdesc, k_pages, v_pages, k_scale, v_scale, page_table));
  for (const void *x : {q, gist_k, gist_v, static_cast<const void *>(n_gists), static_cast<const void *>(own_len),
                        static_cast<const void *>(out), static_cast<const void *>(ws)})
    GSA_TRY(need_ptr(x));
  GSA_TRY(opt_ptr(lse));
  GSA_TRY(opt_ptr(sel_idx));
  GSA_TRY(opt_ptr(sel_score));
  const Layout L = layout(desc, GSA_OP_DECODE, nullptr);
  if (ws_bytes < L.total) return GSA_ERR_WORKSPACE;
  uint32_t *status = reinterpret_cast<uint32_t *>(at(ws, L.status));
  uint32_t *counters = reinterpret_cast<uint32_t *>(at(ws, L.counters));
  float *scores = reinterpret_cast<float *>(at(ws, L.scores));
  int32_t *si = sel_idx ? sel_idx : reinterpret_cast<int32_t *>(at(ws, L.sel_idx));
  float *ss = sel_score ? sel_score : reinterpret_cast<float *>(at(ws, L.sel_score));
  float *part = desc->exclude_unselected ? nullptr : reinterpret_cast<float *>(at(ws, L.part_g));
  int n_prior = 0;
  uint32_t *ready = nullptr;
  if (tail_select_ok(desc)) {
    // as gsa_decode: the scoring selects in its tail and publishes the rows that the unfold's CTAs take
    ready = reinterpret_cast<uint32_t *>(at(ws, L.ready));
    GSA_TRY(run_score(desc, q, gist_k, gist_v, n_gists, 1, desc->n_max, scores, desc->n_max, part, &n_prior, status,
                      stream, counters, reinterpret_cast<uint32_t *>(at(ws, L.unit_counters)), si, ss, ready));
  } else {
    GSA_TRY(run_score(desc, q, gist_k, gist_v, n_gists, 1, desc->n_max, scores, desc->n_max, part, &n_prior, status,
                      stream));
    if (desc->topk > 0)
      GSA_TRY(run_topk(desc->batch * desc->hq, desc->hq, scores, desc->n_max, n_gists, 1, nullptr, desc->topk, nullptr,
                       si, ss, counters, stream));
  }
  return run_paged_unfold(desc, pdesc, q, k_pages, v_pages, k_scale, v_scale, page_table, gist_v, n_gists, own_len, si,
                          ss, part, part ? n_prior : 0, out, lse, L, ws, stream, desc->topk > 0 || ready, ready);
}

gsa_status gsa_paged_gist_step(const gsa_desc *desc, const gsa_pdesc *pdesc, const void *q, const void *k_new,
                               const void *v_new, void *gist_k, void *gist_v, const void *k_pages,
                               const void *v_pages, const float *k_scale, const float *v_scale,
                               const int32_t *page_table, int32_t *n_gists, int32_t *own_len, void *out, float *lse,
                               void *ws, size_t ws_bytes, void *stream) {
  GSA_TRY(check_paged_read(desc, pdesc, k_pages, v_pages, k_scale, v_scale, page_table));
  for (const void *x : {q, k_new, v_new, static_cast<const void *>(gist_k), static_cast<const void *>(gist_v),
                        static_cast<const void *>(n_gists), static_cast<const void *>(own_len),
                        static_cast<const void *>(out), static_cast<const void *>(ws)})
    GSA_TRY(need_ptr(x));
  GSA_TRY(opt_ptr(lse));
  const Layout L = layout(desc, GSA_OP_PAGED, nullptr);
  if (ws_bytes < L.total) return GSA_ERR_WORKSPACE;
  const gsa_desc g = gist_step_desc(desc);
  int n_prior = 0;
  GSA_TRY(gist_step_front(&g, q, k_new, v_new, gist_k, gist_v, n_gists, L, ws, &n_prior, stream));
  const int32_t *n_cur = reinterpret_cast<int32_t *>(at(ws, L.gs_cur));
  const int32_t *n_plus = reinterpret_cast<int32_t *>(at(ws, L.gs_plus));
  GSA_TRY(run_paged_unfold(&g, pdesc, q, k_pages, v_pages, k_scale, v_scale, page_table, gist_v, n_cur, own_len,
                           nullptr, nullptr, reinterpret_cast<float *>(at(ws, L.part_g)), n_prior, out, lse, L, ws,
                           stream, false));
  return launch(k_gist_commit, dim3(cdiv(g.batch, 128)), dim3(128), 0, stream, n_cur, n_plus, n_gists, own_len,
                static_cast<int>(g.batch));
}

}  // extern "C"
