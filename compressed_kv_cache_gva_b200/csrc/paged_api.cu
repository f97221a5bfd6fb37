// C ABI of the paged serving calls: argument validation, kernel selection, workspace
// layout, TMA descriptors and launches.  No allocation, no synchronisation.
#include <stdarg.h>
#include <stdio.h>

#include "common.cuh"
#include "launch.h"
#include "paged.h"

namespace gva {
// defined in api.cu
void set_error_message(const char* msg);
gva_status_t shape_status(const gva_shape_t* shape);
gva_status_t encode_rows(CUtensorMap* m, const void* base, long long rows, int cols, int box_rows,
                         int box_cols, CUtensorMapSwizzle sw);
int device_sms();
}  // namespace gva

namespace {

gva_status_t refuse(gva_status_t s, const char* fmt, ...) {
  char msg[320];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  gva::set_error_message(msg);
  return s;
}

gva_status_t launched(cudaError_t e, const char* what) {
  return e == cudaSuccess ? GVA_OK : refuse(GVA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// No C++ exception (out of host memory in the attribute record) leaves the library.
template <class F>
gva_status_t guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    return refuse(GVA_ERR_CUDA, "out of host memory");
  }
}

bool aligned(const void* p, int n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// One kernel's share of the workspace: piece records, (max, sum) and outputs.
struct Share {
  size_t meta, ml, o, end;
  Share after(size_t at) const { return Share{at + meta, at + ml, at + o, at + end}; }   // (at: a multiple of 256)
};

Share share(size_t metas, size_t slots, size_t rows, size_t d_h) {
  Share s;
  s.meta = 0;
  s.ml = gva::align_up(s.meta + sizeof(int4) * metas, 256);
  s.o = gva::align_up(s.ml + sizeof(float2) * slots * rows, 256);
  s.end = gva::align_up(s.o + sizeof(float) * slots * rows * d_h, 256);
  return s;
}

struct PagedPlan {
  int cols;        // columns of the mma.sync kernel, 0: not launched
  int mma_new;     // most new tokens of a sequence it takes
  int mma_grid;
  enum { kNone, kTc, kSimt } rows;   // the row-block kernel
  int rows_grid;
  Share mma, blk;
  size_t total;
};

bool uses_mma(const gva_shape_t& sh, int page) {
  return !(sh.flags & GVA_FLAG_FMA_PATH) && gva::paged_mma_supported(sh, page);
}
bool uses_tc(const gva_shape_t& sh, int page) {
  return !(sh.flags & GVA_FLAG_FMA_PATH) && gva::paged_tc_supported(sh, page);
}

// Four groups of 16 columns take one CTA per SM.  A long batch of mostly single tokens
// streams faster through two, its few drafts beside it in row blocks: 64 x 1k-8k tokens
// with four new ones from every fourth request 65 us, 77 in one kernel; on 16 x 1k-8k
// 32 and 24 us, with 1 to 4 new tokens each on 64 x 1k-8k 90 and 78 us.  Only where row
// blocks run on tcgen05: with d_h = 32 they would take the CUDA cores, 322 us instead of 82
// for 64 x 6k-8k tokens with four new ones from every fourth request.
bool long_batch(const gva_shape_t& sh, int page, long long max_total) {
  return sh.G == 4 && uses_tc(sh, page) && max_total * sh.G * sh.d_h * 2 >= (96ll << 20);
}

// The shares of the kernels, from 0 on.  cap_B: see the grids.
Share mma_share(const gva_shape_t& sh, int cols, int max_new, int sms, long long max_total, int cap_B,
                PagedPlan* p) {
  const int hpr = sh.H / sh.G;
  p->mma_new = cols / hpr < max_new ? cols / hpr : max_new;
  p->mma_grid = gva::paged_mma_grid(sh, cols, sms, max_total, cap_B);
  return share(sh.B, (size_t)p->mma_grid + sh.B, (size_t)sh.H * p->mma_new, sh.d_h);
}
Share rows_share(const gva_shape_t& sh, bool tc, int n_rows, int max_new, int sms, long long max_total,
                 int cap_B, PagedPlan* p) {
  p->rows_grid = tc ? gva::paged_tc_grid(sh, n_rows, max_new, sms, max_total)
                    : gva::paged_simt_grid(sh, n_rows, sms, max_total, cap_B);
  const size_t g = 2 * (size_t)p->rows_grid;
  return share(g, g, tc ? gva::kPagedTcRows : gva::kPagedSimtRows, sh.d_h);
}
constexpr size_t kPagedHead = 256;   // the status word

// Bytes that serve every call of these heads and types whose B, n_rows, max_new and
// max_total are no larger.  A single plan's bytes do not: fewer new tokens may take the
// split-KV kernel, with a state per CTA and head, where more take row blocks.
size_t most_paged(const gva_shape_t& sh, int page, int n_rows, int max_new, int sms, long long max_total) {
  const int hpr = sh.H / sh.G;
  PagedPlan p{};
  size_t split = 0;
  bool rows = true;
  if (uses_mma(sh, page)) {
    rows = gva::paged_mma_cols(sh, (long long)max_new * hpr) == 0;
    for (int cols = 4; cols <= 16; cols *= 2) {
      if (cols < hpr || (cols == 16 && gva::paged_mma_cols(sh, 16) != 16)) continue;
      const size_t end = mma_share(sh, cols, max_new, sms, max_total, 1, &p).end;
      split = end > split ? end : split;
    }
    const int first16 = 8 / hpr + 1;   // the fewest new tokens that take 16 columns, if any do
    if (first16 <= max_new && gva::paged_mma_cols(sh, (long long)first16 * hpr) == 16 &&
        long_batch(sh, page, max_total))
      rows = true;
  }
  return kPagedHead + split + (rows ? rows_share(sh, uses_tc(sh, page), n_rows, max_new, sms, max_total, 1, &p).end : 0);
}

gva_status_t plan_paged(const gva_shape_t& sh, int page, int n_rows, int max_new, long long max_total,
                        PagedPlan* p) {
  const int sms = gva::device_sms();
  if (sms <= 0) return refuse(GVA_ERR_CUDA, "no CUDA device");
  const int hpr = sh.H / sh.G;
  const bool mma = uses_mma(sh, page), tc = uses_tc(sh, page);
  *p = PagedPlan{};
  p->rows = PagedPlan::kNone;
  if (mma) p->cols = gva::paged_mma_cols(sh, (long long)max_new * hpr);
  if (p->cols == 16 && (long long)n_rows * hpr <= 8ll * sh.B && long_batch(sh, page, max_total)) p->cols = 0;
  if (!p->cols) {
    p->rows = tc ? PagedPlan::kTc : PagedPlan::kSimt;
    if (!tc && !gva::paged_simt_supported(sh))
      return refuse(GVA_ERR_UNSUPPORTED, "no paged attention kernel for H=%d G=%d d_h=%d d_r=%d", sh.H,
                    sh.G, sh.d_h, sh.d_r);
    // Sequences with few new tokens go to the mma.sync kernel, unless every one of
    // them brings max_new (the rows then fill all of n_rows).
    if (mma && (long long)sh.B * max_new > n_rows) p->cols = hpr <= 4 ? 4 : 8;
  }
  p->total = kPagedHead;
  if (p->cols) {
    p->mma = mma_share(sh, p->cols, max_new, sms, max_total, sh.B, p).after(p->total);
    p->total = p->mma.end;
  }
  if (p->rows != PagedPlan::kNone) {
    p->blk = rows_share(sh, tc, n_rows, max_new, sms, max_total, sh.B, p).after(p->total);
    p->total = p->blk.end;
  }
  return GVA_OK;
}

gva_status_t paged_sizes(const gva_shape_t* sh, int page, int n_rows, int max_new, long long max_total) {
  gva_status_t s = gva::shape_status(sh);
  if (s != GVA_OK) return s;
  if (page < 1 || page > (1 << 20)) return refuse(GVA_ERR_INVALID_ARG, "page_size=%d outside [1, 2^20]", page);
  if (n_rows < 0 || (long long)n_rows * sh->H >= (1ll << 31))
    return refuse(GVA_ERR_INVALID_ARG, "n_rows=%d: n_rows * H must be in [0, 2^31)", n_rows);
  if (max_new < 1) return refuse(GVA_ERR_INVALID_ARG, "max_query_len=%d < 1", max_new);
  if (max_total < 0 || max_total >= (1ll << 31))
    return refuse(GVA_ERR_INVALID_ARG, "max_total_tokens=%lld outside [0, 2^31)", max_total);
  return GVA_OK;
}

gva_status_t paged_attention(const gva_shape_t* shp, int page, const float* q_abs, const void* V,
                             const void* KR, int64_t num_slots, const int32_t* table, int max_pages,
                             int64_t table_stride, const int32_t* q_start, const int32_t* seq_len,
                             int n_rows, int max_new, int64_t max_total, void* out, float* lse,
                             void* workspace, size_t ws_bytes, cudaStream_t st) {
  gva_status_t s = paged_sizes(shp, page, n_rows, max_new, max_total);
  if (s != GVA_OK) return s;
  const gva_shape_t& sh = *shp;
  if (sh.B == 0 || n_rows == 0) return GVA_OK;
  if (max_new > n_rows) max_new = n_rows;
  if (!q_abs || !V || !table || !q_start || !seq_len || !out || !workspace || (sh.d_r > 0 && !KR))
    return refuse(GVA_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned(q_abs, 16) || !aligned(V, 16) || (sh.d_r > 0 && !aligned(KR, 16)) || !aligned(out, 16) ||
      !aligned(lse, 16) || !aligned(workspace, 16))
    return refuse(GVA_ERR_INVALID_ARG, "pointers must be 16-byte aligned");
  if (!aligned(table, 4) || !aligned(q_start, 4) || !aligned(seq_len, 4))
    return refuse(GVA_ERR_INVALID_ARG, "index arrays must be 4-byte aligned");
  if (num_slots < 1 || num_slots >= (1ll << 31) - 512 || num_slots % page)
    return refuse(GVA_ERR_INVALID_ARG, "num_slots=%lld must be a multiple of page_size=%d in [1, 2^31 - 512)",
                  (long long)num_slots, page);
  if (max_pages < 1 || table_stride < max_pages)
    return refuse(GVA_ERR_INVALID_ARG, "max_pages=%d, table_stride=%lld", max_pages, (long long)table_stride);
  const int e = sh.cache_dtype == GVA_F32 ? 4 : 2;
  if ((sh.G * sh.d_h * e) % 16 || (sh.d_r * e) % 16)
    return refuse(GVA_ERR_INVALID_ARG, "cache rows must be multiples of 16 bytes (G*d_h*elt=%d, d_r*elt=%d)",
                  sh.G * sh.d_h * e, sh.d_r * e);
  PagedPlan p;
  if ((s = plan_paged(sh, page, n_rows, max_new, max_total, &p)) != GVA_OK) return s;
  if (ws_bytes < p.total) return refuse(GVA_ERR_WORKSPACE, "workspace %zu bytes < required %zu", ws_bytes, p.total);

  gva::PagedArgs a{};
  a.B = sh.B; a.H = sh.H; a.G = sh.G; a.hpr = sh.H / sh.G; a.d_h = sh.d_h; a.d_r = sh.d_r;
  a.page = page; a.max_pages = max_pages; a.table_stride = table_stride;
  a.num_pages = (int)(num_slots / page);
  a.num_slots = (int)num_slots;
  a.n_rows = n_rows; a.max_new = max_new;
  a.q_abs = q_abs; a.V = V; a.KR = KR; a.table = table; a.q_start = q_start; a.seq_len = seq_len;
  a.out = out; a.lse = lse; a.out_bf16 = sh.out_dtype == GVA_BF16;
  a.wide = aligned(out, 32) && aligned(workspace, 32);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.status = reinterpret_cast<int*>(ws);

  // Boxes of cache rows: the largest power of two that divides the page, up to the
  // tile, so that a box never crosses a page.
  auto maps = [&](int tile, gva::PagedArgs& k, CUtensorMap* tv, CUtensorMap* tk) -> gva_status_t {
    k.box_log2 = 0;
    while ((2 << k.box_log2) <= tile && page % (2 << k.box_log2) == 0) ++k.box_log2;
    k.box = 1 << k.box_log2;
    const int vw = sh.d_h < 64 ? sh.d_h : 64;
    gva_status_t r = gva::encode_rows(tv, V, num_slots, sh.G * sh.d_h, k.box, vw,
                                      vw == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
    if (r != GVA_OK) return r;
    *tk = *tv;
    if (sh.d_r == 0) return GVA_OK;
    const int drp = sh.d_r <= 16 ? 16 : 32;
    return gva::encode_rows(tk, KR, num_slots, sh.d_r, k.box, drp,
                            drp == 16 ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_64B);
  };
  auto place = [&](gva::PagedArgs& k, const Share& w) {
    k.meta = reinterpret_cast<int4*>(ws + w.meta);
    k.part_ml = reinterpret_cast<float2*>(ws + w.ml);
    k.part_o = reinterpret_cast<float*>(ws + w.o);
  };

  // The descriptors of both kernels are made before the first launch.
  gva::PagedArgs am = a, ar = a;
  CUtensorMap mv{}, mk{}, rv{}, rk{};
  am.lo_rows = 0;
  am.hi_rows = p.cols;
  am.flag_errors = 1;
  am.grid = p.mma_grid;
  if (p.cols && (s = maps(gva::paged_mma_tile(sh), am, &mv, &mk)) != GVA_OK) return s;
  ar.lo_rows = p.cols;
  ar.hi_rows = 0x7fffffff;
  ar.flag_errors = p.cols ? 0 : 1;
  ar.grid = p.rows_grid;
  if (p.rows == PagedPlan::kTc && (s = maps(gva::paged_tc_tile(sh), ar, &rv, &rk)) != GVA_OK) return s;

  const bool tc = p.rows == PagedPlan::kTc, rows = p.rows != PagedPlan::kNone;
  if (p.cols) {
    place(am, p.mma);
    if ((s = launched(gva::launch_paged_mma(sh, am, p.cols, mv, mk, st), "paged attention launch")) != GVA_OK)
      return s;
  }
  if (rows) {
    place(ar, p.blk);
    ar.beside = p.cols != 0;
    if ((s = launched(tc ? gva::launch_paged_tc(sh, ar, rv, rk, st) : gva::launch_paged_simt(sh, ar, st),
                      "paged attention launch")) != GVA_OK)
      return s;
  }
  am.max_new = p.mma_new;   // heads of a partial: H * mma_new
  return launched(gva::launch_paged_merge(p.cols ? &am : nullptr, rows ? &ar : nullptr,
                                          tc ? gva::kPagedTcRows : gva::kPagedSimtRows, st),
                  "paged merge launch");
}

}  // namespace

extern "C" {

gva_status_t gva_plan_pages(int32_t B, int32_t page_size, int32_t num_pages, int32_t max_pages,
                            int64_t table_stride, int32_t max_new_tokens, const int32_t* kept_len,
                            const int32_t* n_new, const int32_t* held_in, int32_t* held_out,
                            int32_t* free_pages, const int32_t* free_count_in,
                            int32_t* free_count_out, int32_t* block_table, int32_t* q_start,
                            int32_t* seq_len, int32_t* n_granted, int32_t* slot, int32_t* pos,
                            int32_t* err_flag, void* stream) {
  if (B < 0 || B > gva::kMaxBatch) return refuse(GVA_ERR_INVALID_ARG, "B=%d outside [0, %d]", B, gva::kMaxBatch);
  if (page_size < 1 || num_pages < 1 || (long long)page_size * num_pages >= (1ll << 31))
    return refuse(GVA_ERR_INVALID_ARG, "page_size=%d, num_pages=%d: need >= 1 and a product below 2^31",
                  page_size, num_pages);
  if (max_pages < 1 || table_stride < max_pages || (long long)page_size * max_pages >= (1ll << 31))
    return refuse(GVA_ERR_INVALID_ARG, "max_pages=%d, table_stride=%lld: need 1 <= max_pages <= table_stride "
                  "and page_size * max_pages below 2^31", max_pages, (long long)table_stride);
  if (max_new_tokens < 0) return refuse(GVA_ERR_INVALID_ARG, "max_new_tokens=%d < 0", max_new_tokens);
  if (!free_pages || !free_count_in || !free_count_out || !q_start || (max_new_tokens > 0 && (!slot || !pos)) ||
      (B > 0 && (!kept_len || !n_new || !held_in || !held_out || !block_table || !seq_len || !n_granted)))
    return refuse(GVA_ERR_INVALID_ARG, "a required pointer is NULL");
  const void* all[] = {kept_len, n_new, held_in, held_out, free_pages, free_count_in, free_count_out,
                       block_table, q_start, seq_len, n_granted, slot, pos, err_flag};
  for (const void* q : all)
    if (!aligned(q, 4)) return refuse(GVA_ERR_INVALID_ARG, "pointers must be 4-byte aligned");
  gva::PlanArgs a{};
  a.B = B; a.page = page_size; a.max_pages = max_pages; a.num_pages = num_pages; a.max_new = max_new_tokens;
  a.table_stride = table_stride;
  a.kept_len = kept_len; a.n_new = n_new; a.held_in = held_in; a.held_out = held_out;
  a.free_pages = free_pages; a.free_count_in = free_count_in; a.free_count_out = free_count_out;
  a.table = block_table; a.q_start = q_start; a.seq_len = seq_len; a.n_granted = n_granted;
  a.slot = slot; a.pos = pos; a.err_flag = err_flag;
  return guarded([&] { return launched(gva::launch_plan_pages(a, static_cast<cudaStream_t>(stream)), "page plan launch"); });
}

size_t gva_paged_workspace_size(const gva_shape_t* shape, int32_t page_size, int32_t n_rows,
                                int32_t max_query_len, int64_t max_total_tokens) {
  if (paged_sizes(shape, page_size, n_rows, max_query_len, max_total_tokens) != GVA_OK) return 0;
  if (shape->B == 0 || n_rows == 0) return 256;
  PagedPlan p;
  const int most = max_query_len < n_rows ? max_query_len : n_rows;
  if (plan_paged(*shape, page_size, n_rows, most, max_total_tokens, &p) != GVA_OK) return 0;
  return most_paged(*shape, page_size, n_rows, most, gva::device_sms(), max_total_tokens);
}

gva_status_t gva_paged_attention(const gva_shape_t* shape, int32_t page_size, const float* q_abs,
                                 const void* V_cache, const void* kr_cache, int64_t num_slots,
                                 const int32_t* block_table, int32_t max_pages,
                                 int64_t table_stride, const int32_t* q_start,
                                 const int32_t* seq_len, int32_t n_rows, int32_t max_query_len,
                                 int64_t max_total_tokens, void* out, float* lse, void* workspace,
                                 size_t ws_bytes, void* stream) {
  return guarded([&] {
    return paged_attention(shape, page_size, q_abs, V_cache, kr_cache, num_slots, block_table, max_pages,
                           table_stride, q_start, seq_len, n_rows, max_query_len, max_total_tokens, out,
                           lse, workspace, ws_bytes, static_cast<cudaStream_t>(stream));
  });
}

gva_status_t gva_verify_draft(int32_t B, int32_t vocab, int32_t n_rows, const int32_t* tokens,
                              const int32_t* q_start, int32_t probs_dtype,
                              const void* target_probs, int64_t target_stride,
                              const void* draft_probs, int64_t draft_stride,
                              const float* u_accept, const float* u_sample, int32_t* out_tokens,
                              int32_t* n_accepted, const int32_t* seq_len, int32_t* kept_len,
                              int32_t* err_flag, void* stream) {
  if (B < 0 || B > 65535) return refuse(GVA_ERR_INVALID_ARG, "B=%d outside [0, 65535]", B);
  if (vocab < 1 || vocab > (1 << 30)) return refuse(GVA_ERR_INVALID_ARG, "vocab=%d outside [1, 2^30]", vocab);
  // (a block's loop over a request's rows counts up to its width past the last)
  if (n_rows < 0 || n_rows > INT32_MAX - 1024)
    return refuse(GVA_ERR_INVALID_ARG, "n_rows=%d outside [0, 2^31 - 1025]", n_rows);
  if (probs_dtype != GVA_F32 && probs_dtype != GVA_BF16)
    return refuse(GVA_ERR_INVALID_ARG, "probs_dtype must be GVA_F32 or GVA_BF16");
  if (target_stride < vocab || (draft_probs && draft_stride < vocab))
    return refuse(GVA_ERR_INVALID_ARG, "row strides %lld, %lld below vocab=%d", (long long)target_stride,
                  (long long)draft_stride, vocab);
  if (B == 0) return GVA_OK;
  if (!q_start || !n_accepted || !u_sample ||
      (n_rows > 0 && (!tokens || !target_probs || !u_accept || !out_tokens)))
    return refuse(GVA_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!seq_len != !kept_len) return refuse(GVA_ERR_INVALID_ARG, "seq_len and kept_len go together");
  const void* words[] = {tokens, q_start, u_accept, u_sample, out_tokens, n_accepted, seq_len, kept_len, err_flag};
  for (const void* q : words)
    if (!aligned(q, 4)) return refuse(GVA_ERR_INVALID_ARG, "pointers must be 4-byte aligned");
  const int e = probs_dtype == GVA_F32 ? 4 : 2;
  if (!aligned(target_probs, e) || !aligned(draft_probs, e))
    return refuse(GVA_ERR_INVALID_ARG, "probabilities must be aligned to their type");
  // the CTAs of a request read its tokens at their own pace while the first writes the result
  const uintptr_t t0 = reinterpret_cast<uintptr_t>(tokens), o0 = reinterpret_cast<uintptr_t>(out_tokens);
  if (n_rows > 0 && t0 < o0 + 4ull * n_rows && o0 < t0 + 4ull * n_rows)
    return refuse(GVA_ERR_INVALID_ARG, "out_tokens must not overlap tokens");
  const int sms = gva::device_sms();
  if (sms <= 0) return refuse(GVA_ERR_CUDA, "no CUDA device");
  gva::VerifyArgs a{};
  a.B = B; a.vocab = vocab; a.n_rows = n_rows; a.tokens = tokens; a.q_start = q_start;
  a.target = target_probs; a.draft = draft_probs; a.target_stride = target_stride; a.draft_stride = draft_stride;
  a.u_accept = u_accept; a.u_sample = u_sample; a.out_tokens = out_tokens; a.n_accepted = n_accepted;
  a.seq_len = seq_len; a.kept_len = kept_len; a.err_flag = err_flag;
  return guarded([&] {
    return launched(gva::launch_verify(a, probs_dtype == GVA_BF16, sms, static_cast<cudaStream_t>(stream)),
                    "draft verification launch");
  });
}

}  // extern "C"
