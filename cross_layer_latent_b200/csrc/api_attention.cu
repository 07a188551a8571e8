// api_attention.cu -- the extern "C" entry points of the attention operators
// (include/li.h, "attention over the selected tokens"): argument checks,
// workspace layout and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "attention.h"
#include "ctx.h"
#include "internal.h"
#include "sm100.cuh"

using namespace li;

namespace {

// Status word at 0 and completion counter at 64, as in every workspace.
constexpr size_t kAttnHeader = 256;

li_status check_device(li_ctx* c, const char* what) {
  int dev = -1;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(c, e, what);
  if (dev != c->device)
    return fail(c, LI_ERR_ARG, "%s: the context's device (%d) must be the current device (%d)", what, c->device, dev);
  return LI_OK;
}

li_status check_type(li_ctx* c, li_dtype d, const char* what) {
  if (d != LI_F32 && d != LI_BF16) return fail(c, LI_ERR_DTYPE, "%s: F32 or BF16 only (got %d)", what, static_cast<int>(d));
  return LI_OK;
}

li_status check_attn_ws(li_ctx* c, const void* ws, size_t bytes, size_t need, const char* what) {
  if (!ws) return fail(c, LI_ERR_WORKSPACE, "%s: workspace is NULL", what);
  if (!aligned(ws, 256)) return fail(c, LI_ERR_WORKSPACE, "%s: workspace not 256-byte aligned", what);
  if (bytes < need) return fail(c, LI_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", what, bytes, need);
  return LI_OK;
}

// Checks a row transform for rows of `dim` elements and copies it to *out
// without the fields of parts that are switched off, which the kernels then
// need not tell from parts that are on (an off part is an empty range);
// *chunked tells whether its ranges suit the wide path (whole chunks of 8).
li_status check_transform(li_ctx* c, const li_row_transform& tf, int dim, li_row_transform* out, bool* chunked, const char* what) {
  memset(out, 0, sizeof(*out));
  out->norm = LI_NORM_NONE;
  if (tf.norm != LI_NORM_NONE && tf.norm != LI_NORM_RMS && tf.norm != LI_NORM_LAYER)
    return fail(c, LI_ERR_ARG, "%s: unknown norm %d", what, static_cast<int>(tf.norm));
  if (tf.norm != LI_NORM_NONE) {
    if (tf.norm_dim < 1 || tf.norm_offset < 0 || tf.norm_offset > dim - tf.norm_dim)
      return fail(c, LI_ERR_SHAPE, "%s: norm range of %d at %d outside the row of %d", what, tf.norm_dim, tf.norm_offset, dim);
    if (!(tf.eps >= 0.f) || !std::isfinite(tf.eps)) return fail(c, LI_ERR_ARG, "%s: eps must be finite and >= 0", what);
    if (!aligned(tf.gamma, 4) || !aligned(tf.beta, 4)) return fail(c, LI_ERR_ALIGN, "%s: gamma and beta must be 4-byte aligned", what);
    if (tf.norm_offset % 8 || tf.norm_dim % 8) *chunked = false;
    out->norm = tf.norm;
    out->norm_offset = tf.norm_offset;
    out->norm_dim = tf.norm_dim;
    out->gamma = tf.gamma;
    out->beta = tf.beta;
    out->eps = tf.eps;
  }
  if (tf.rope_dim != 0) {
    if (tf.rope_dim < 2 || tf.rope_dim % 2 || tf.rope_offset < 0 || tf.rope_offset > dim - tf.rope_dim)
      return fail(c, LI_ERR_SHAPE, "%s: rotary range of %d at %d must be even and inside the row of %d", what, tf.rope_dim,
                  tf.rope_offset, dim);
    if (tf.rope_halves != 0 && tf.rope_halves != 1) return fail(c, LI_ERR_ARG, "%s: rope_halves must be 0 or 1", what);
    if (!tf.inv_freq) return fail(c, LI_ERR_ARG, "%s: inv_freq is NULL", what);
    if (!aligned(tf.inv_freq, 4)) return fail(c, LI_ERR_ALIGN, "%s: inv_freq must be 4-byte aligned", what);
    if (tf.rope_offset % 8 || tf.rope_dim % 8) *chunked = false;
    if (tf.rope_halves && tf.rope_dim % 16) *chunked = false;
    out->rope_offset = tf.rope_offset;
    out->rope_dim = tf.rope_dim;
    out->rope_halves = tf.rope_halves;
    out->inv_freq = tf.inv_freq;
  }
  return LI_OK;
}

li_status check_paged(li_ctx* c, const li_paged_cache* p, const char* what) {
  if (!p) return fail(c, LI_ERR_ARG, "%s: cache is NULL", what);
  if (!p->data || !p->page_table || !p->lengths) return fail(c, LI_ERR_ARG, "%s: cache data, page_table and lengths must be non-NULL", what);
  li_status s = check_type(c, p->dtype, what);
  if (s != LI_OK) return s;
  if (p->batch < 1 || p->n_pages < 1 || p->page_size < 1 || p->max_pages < 1 || p->dim < 1)
    return fail(c, LI_ERR_SHAPE, "%s: batch, n_pages, page_size, max_pages and dim must be >= 1", what);
  if (static_cast<int64_t>(p->n_pages) * p->page_size >= (int64_t(1) << 31) ||
      static_cast<int64_t>(p->max_pages) * p->page_size >= (int64_t(1) << 31))
    return fail(c, LI_ERR_SHAPE, "%s: n_pages and max_pages times page_size must be < 2^31", what);
  if (static_cast<int64_t>(p->dim) * elt_bytes(p->dtype) % 16)
    return fail(c, LI_ERR_SHAPE, "%s: rows of %d elements are not a multiple of 16 bytes", what, p->dim);
  if (!aligned(p->data, 16)) return fail(c, LI_ERR_ALIGN, "%s: cache data not 16-byte aligned", what);
  if (!aligned(p->page_table, 4) || !aligned(p->lengths, 4))
    return fail(c, LI_ERR_ALIGN, "%s: page_table and lengths must be 4-byte aligned", what);
  return LI_OK;
}

li_status norm_rope(li_ctx* c, const li_head_rows* sets, int n_sets, li_dtype dtype, int64_t n_tok, const int32_t* pos,
                    cudaStream_t st) {
  const char* what = "li_norm_rope";
  if (!sets || n_sets < 1 || n_sets > kMaxRowSets)
    return fail(c, LI_ERR_ARG, "%s: need 1 to %d tensors (got %d)", what, kMaxRowSets, n_sets);
  li_status s = check_type(c, dtype, what);
  if (s != LI_OK) return s;
  if (n_tok < 0) return fail(c, LI_ERR_SHAPE, "%s: n_tok must be >= 0", what);
  NormRopeArgs a;
  memset(&a, 0, sizeof(a));
  bool vec = true;
  int max_dim = 0;
  int64_t heads = 0;
  const size_t eb = static_cast<size_t>(elt_bytes(dtype));
  for (int i = 0; i < n_sets; ++i) {
    const li_head_rows& r = sets[i];
    if (n_tok > 0 && (!r.x || !r.out)) return fail(c, LI_ERR_ARG, "%s: x and out must be non-NULL", what);
    if (r.H < 1 || r.dim < 1 || r.dim > kMaxRowDim)
      return fail(c, LI_ERR_SHAPE, "%s: need H >= 1 and dim in [1, %d]", what, kMaxRowDim);
    if (!aligned(r.x, eb) || !aligned(r.out, eb)) return fail(c, LI_ERR_ALIGN, "%s: x and out must be aligned to their elements", what);
    a.set[i] = r;
    if ((s = check_transform(c, r.tf, r.dim, &a.set[i].tf, &vec, what)) != LI_OK) return s;
    if (n_tok > 0 && r.tf.rope_dim && !pos) return fail(c, LI_ERR_ARG, "%s: a rotation needs pos", what);
    if (r.dim % 8 || !aligned(r.x, 16) || !aligned(r.out, 16) || r.tok_stride % 8 || r.head_stride % 8 ||
        r.out_tok_stride % 8 || r.out_head_stride % 8)
      vec = false;
    max_dim = std::max(max_dim, r.dim);
    heads += r.H;
  }
  if (pos && !aligned(pos, 4)) return fail(c, LI_ERR_ALIGN, "%s: pos must be 4-byte aligned", what);
  if (heads > 65535) return fail(c, LI_ERR_SHAPE, "%s: more than 65535 heads", what);
  if (n_tok == 0) return LI_OK;
  a.n_sets = n_sets;
  a.pos = pos;
  const NormRopePlan plan = plan_norm_rope(a.set, n_sets, vec, max_dim);
  for (int i = 0; i < n_sets; ++i) {
    a.tasks += (sets[i].H + plan.rows - 1) / plan.rows;
    a.tab_stride = std::max(a.tab_stride, (a.set[i].tf.rope_dim / 2 + 1) / 2 * 2);
  }
  // A block takes all of a token's tasks (its angles once) when the tokens
  // alone fill the GPU, else one a warp.
  a.per_block = n_tok < 4 * c->num_sms ? std::min(a.tasks, plan.warps) : a.tasks;
  a.blocks = (a.tasks + a.per_block - 1) / a.per_block;
  const int64_t grid = n_tok * a.blocks;
  if (grid >= (int64_t(1) << 31)) return fail(c, LI_ERR_SHAPE, "%s: too many tokens (%lld)", what, static_cast<long long>(n_tok));
  if ((s = check_device(c, what)) != LI_OK) return s;
  (void)cudaGetLastError();
  Launch L(c, st, "norm_rope", static_cast<int>(grid), 32 * plan.warps, 0);
  const cudaError_t e = launch_norm_rope(a, dtype, plan, grid, st);
  L.done();
  return e == cudaSuccess ? LI_OK : cuda_fail(c, e, "norm_rope launch");
}

li_status append_paged(li_ctx* c, const li_paged_cache* cache, const void* x, int T, int64_t tok_stride,
                       const li_row_transform* tf, const int32_t* start, const int32_t* n_new, void* ws, size_t ws_bytes,
                       cudaStream_t st) {
  const char* what = "li_append_paged";
  li_status s = check_paged(c, cache, what);
  if (s != LI_OK) return s;
  if (T < 1) return fail(c, LI_ERR_SHAPE, "%s: T must be >= 1", what);
  if (!x) return fail(c, LI_ERR_ARG, "%s: x is NULL", what);
  if (static_cast<int64_t>(cache->batch) * T >= (int64_t(1) << 31)) return fail(c, LI_ERR_SHAPE, "%s: batch * T too large", what);
  if (cache->dim > kMaxRowDim) return fail(c, LI_ERR_SHAPE, "%s: dim must be <= %d", what, kMaxRowDim);
  const int eb = elt_bytes(cache->dtype);
  const bool one = static_cast<int64_t>(cache->batch) * T == 1;   // a single row has no stride to speak of
  if (!aligned(x, 16) || (!one && tok_stride * eb % 16)) return fail(c, LI_ERR_ALIGN, "%s: rows of x must be 16-byte aligned", what);
  if (!aligned(start, 4) || !aligned(n_new, 4)) return fail(c, LI_ERR_ALIGN, "%s: start and n_new must be 4-byte aligned", what);
  for (const int32_t* p : {start, n_new})
    if (p && p != cache->lengths && p < cache->lengths + cache->batch && cache->lengths < p + cache->batch)
      return fail(c, LI_ERR_ARG, "%s: start and n_new may be the lengths, but not overlap them otherwise", what);
  AppendPagedArgs a;
  memset(&a, 0, sizeof(a));
  bool vec = cache->dim % 8 == 0;
  if (tf && (s = check_transform(c, *tf, cache->dim, &a.tf, &vec, what)) != LI_OK) return s;
  vec = vec && append_in_chunks(a.tf, cache->dim);
  if ((s = check_attn_ws(c, ws, ws_bytes, kAttnHeader, what)) != LI_OK) return s;
  if ((s = check_device(c, what)) != LI_OK) return s;
  a.x = x;
  a.tok_stride = tok_stride;
  a.data = cache->data;
  a.page_table = cache->page_table;
  a.lengths = cache->lengths;
  a.start = start == cache->lengths ? nullptr : start;   // the lengths themselves: they are read before they advance
  a.n_new = n_new;
  a.lengths_last = !a.start || n_new == cache->lengths;
  a.batch = cache->batch;
  a.T = T;
  a.n_pages = cache->n_pages;
  a.page_size = cache->page_size;
  a.max_pages = cache->max_pages;
  a.dim = cache->dim;
  a.done = at<unsigned int>(ws, 64);
  a.status = at<int>(ws, 0);
  (void)cudaGetLastError();
  Launch L(c, st, "append_paged", 0, 128, 0);
  const cudaError_t e = launch_append_paged(a, cache->dtype, vec, c->num_sms, st);
  L.done();
  return e == cudaSuccess ? LI_OK : cuda_fail(c, e, "append_paged launch");
}

li_status latent_mma(li_ctx* c, const li_paged_cache* cache, const void* q, int T, int H, int d_v, float scale,
                     const int32_t* q_pos, const int32_t* sel, int k, void* out, float* lse, void* ws, cudaStream_t st) {
  const char* what = "li_latent_attention";
  LatentMmaArgs a;
  memset(&a, 0, sizeof(a));
  a.data = cache->data;
  a.page_table = cache->page_table;
  a.lengths = cache->lengths;
  a.q_pos = q_pos;
  a.sel = sel;
  a.out = out;
  a.lse = lse;
  a.status = at<int>(ws, 0);
  a.cuts = at<int4>(ws, kAttnHeader);
  a.part_ml = at<float>(ws, kAttnHeader + up256(static_cast<size_t>(c->num_sms) * sizeof(int4)));
  a.part_o = a.part_ml + static_cast<size_t>(c->num_sms) * 2 * 64 * 2;
  a.part_stride = latent_part_stride(d_v);
  a.wait_ns = c->wait_ns;
  a.scale_log2 = scale * 1.44269504089f;
  a.seqs = sel ? cache->batch * T : cache->batch;
  a.rows = sel ? H : T * H;
  a.T = T;
  a.H = H;
  a.k = k;
  a.dim = cache->dim;
  a.d_v = d_v;
  a.n_pages = cache->n_pages;
  a.page_size = cache->page_size;
  a.max_pages = cache->max_pages;
  // whole boxes of rows where a page holds them (the 128-byte swizzle repeats every 8 rows); selected rows come
  // one by one
  a.box = sel ? 0 : 64;
  while (a.box && cache->page_size % a.box) a.box /= 2;
  if (a.box < 8) a.box = 0;
  while ((1 << a.box_shift) < a.box) ++a.box_shift;
  if (!latent_mma_layout(&a, c->num_sms, c->max_smem_optin))
    return fail(c, LI_ERR_UNSUPPORTED, "%s: operands too large for shared memory (dim %d)", what, a.dim);
  const cuuint64_t row_bytes = static_cast<cuuint64_t>(a.dim) * 2;
  const cuuint64_t qdims[3] = {static_cast<cuuint64_t>(a.dim), static_cast<cuuint64_t>(a.rows), static_cast<cuuint64_t>(a.seqs)};
  const cuuint64_t qstr[2] = {row_bytes, row_bytes * a.rows};
  const cuuint32_t qbox[3] = {64, static_cast<cuuint32_t>(a.N), 1};
  li_status s = encode_map(c, &a.map_q, LI_BF16, 3, const_cast<void*>(q), qdims, qstr, qbox, 128);
  if (s != LI_OK) return s;
  if (a.box) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.dim), static_cast<cuuint64_t>(cache->n_pages) * cache->page_size};
    const cuuint64_t str[1] = {row_bytes};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(a.box)};
    if ((s = encode_map(c, &a.map_box, LI_BF16, 2, cache->data, dims, str, box, 128)) != LI_OK) return s;
  }
  (void)cudaGetLastError();
  {
    Launch L(c, st, "latent_attn", a.grid, 448, static_cast<int>(a.smem_bytes));
    const cudaError_t e = launch_latent_mma(a, st);
    L.done();
    if (e != cudaSuccess) return cuda_fail(c, e, "latent attention launch");
  }
  if (a.n_cuts == 0) return LI_OK;
  Launch L(c, st, "latent_join", a.n_cuts, 128, 0);
  const cudaError_t e = launch_latent_join(a, st);
  L.done();
  return e == cudaSuccess ? LI_OK : cuda_fail(c, e, "latent attention join launch");
}

li_status latent_attention(li_ctx* c, const li_paged_cache* cache, const void* q, int T, int H, int d_v, float scale,
                           const int32_t* q_pos, const int32_t* sel, int k, void* out, float* lse, void* ws,
                           size_t ws_bytes, cudaStream_t st) {
  const char* what = "li_latent_attention";
  li_status s = check_paged(c, cache, what);
  if (s != LI_OK) return s;
  if (T < 1 || H < 1) return fail(c, LI_ERR_SHAPE, "%s: T and H must be >= 1", what);
  if (cache->dim > 576 || d_v < 1 || d_v > cache->dim || d_v > 512)
    return fail(c, LI_ERR_SHAPE, "%s: need dim <= 576 and d_v in [1, min(dim, 512)] (dim %d, d_v %d)", what, cache->dim, d_v);
  if (!q || !out) return fail(c, LI_ERR_ARG, "%s: q and out must be non-NULL", what);
  if (sel && k < 1) return fail(c, LI_ERR_SHAPE, "%s: k must be >= 1 with sel", what);
  if (!std::isfinite(scale)) return fail(c, LI_ERR_ARG, "%s: scale must be finite", what);
  if (static_cast<double>(cache->batch) * T * H >= 2147483648.0) return fail(c, LI_ERR_SHAPE, "%s: batch * T * H too large", what);
  if (!aligned(q, 16) || !aligned(out, elt_bytes(cache->dtype)) || !aligned(lse, 4) || !aligned(sel, 4) || !aligned(q_pos, 4))
    return fail(c, LI_ERR_ALIGN, "%s: q must be 16-byte aligned, the other tensors to their elements", what);
  if ((s = check_attn_ws(c, ws, ws_bytes, li_attention_workspace_bytes(c, H, d_v), what)) != LI_OK) return s;
  if ((s = check_device(c, what)) != LI_OK) return s;
  if (cache->dtype == LI_BF16)
    return latent_mma(c, cache, q, T, H, d_v, scale, q_pos, sel, k, out, lse, ws, st);
  LatentAttnArgs a;
  memset(&a, 0, sizeof(a));
  a.q = static_cast<const float*>(q);
  a.data = static_cast<const float*>(cache->data);
  a.page_table = cache->page_table;
  a.lengths = cache->lengths;
  a.q_pos = q_pos;
  a.sel = sel;
  a.out = static_cast<float*>(out);
  a.lse = lse;
  a.status = at<int>(ws, 0);
  a.batch = cache->batch;
  a.T = T;
  a.H = H;
  a.k = k;
  a.dim = cache->dim;
  a.d_v = d_v;
  a.n_pages = cache->n_pages;
  a.page_size = cache->page_size;
  a.max_pages = cache->max_pages;
  a.scale = scale;
  (void)cudaGetLastError();
  Launch L(c, st, "latent_attn_rows", 0, 256, 0);
  const cudaError_t e = launch_latent_attn_rows(a, st);
  L.done();
  return e == cudaSuccess ? LI_OK : cuda_fail(c, e, "latent attention launch");
}

// A tensor of rows [tokens][heads][d] as a map with boxes of `rows` rows and 64
// columns (heads = 0: no head dimension).  Strides of dimensions of one
// element are free, so they are set to something the map takes.
li_status rows_map(li_ctx* c, CUtensorMap* m, const void* base, int rows, int d, int heads, int tokens, int64_t head_stride,
                   int64_t tok_stride) {
  const cuuint64_t hs = static_cast<cuuint64_t>(heads > 1 ? head_stride : (d + 7) / 8 * 8) * 2;
  const cuuint64_t ts = static_cast<cuuint64_t>(tokens > 1 ? tok_stride : (d + 7) / 8 * 8) * 2;
  if (heads == 0) {
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(tokens)}, str[1] = {ts};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(rows)};
    return encode_map(c, m, LI_BF16, 2, const_cast<void*>(base), dims, str, box, 128);
  }
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens)};
  const cuuint64_t str[2] = {hs, ts};
  const cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(rows)};
  return encode_map(c, m, LI_BF16, 3, const_cast<void*>(base), dims, str, box, 128);
}

li_status prompt_mma(li_ctx* c, const li_prompt& p, void* out, float* lse, void* ws, cudaStream_t st) {
  const char* what = "li_prompt_attention";
  PromptMmaArgs a;
  memset(&a, 0, sizeof(a));
  a.cu_q = p.cu_q;
  a.cu_k = p.cu_k;
  a.out = out;
  a.lse = lse;
  a.status = at<int>(ws, 0);
  a.next_unit = at<unsigned int>(ws, 128);
  a.done = at<unsigned int>(ws, 132);
  a.wait_ns = c->wait_ns;
  // a scale of 0 makes every weight equal; the smallest steps of the scores do the same and keep -inf apart
  a.scale_log2 = std::max(std::fabs(p.scale) * 1.44269504089f, 1e-30f);
  a.negate = p.scale < 0.f;
  a.causal = p.causal != 0;
  a.wide_out = aligned(out, 32) && p.d_v % 16 == 0;
  a.batch = p.batch;
  a.H = p.H;
  a.total_q = p.total_q;
  a.total_k = p.total_k;
  a.max_q = p.max_q;
  a.d_nope = p.d_nope;
  a.d_rope = p.d_rope;
  a.d_v = p.d_v;
  // Pairs of CTAs halve what an SM reads of keys and values, but their units are twice as many queries and take longer
  // to begin and end.  Measured at d 192/128, 20 calls in a row (single CTAs, pairs): 8 sequences of up to 257 x 16 heads
  // 18, 26 us; 4 of 1500 to 2048 x 32 170, 183; 4 of 2048 x 32 197, 203; 4 of 1000 to 4096 x 16 185, 208; 1 of 4096 x 32
  // 203, 184; 1 of 8192 x 32 637, 605.  The rule knows max_q alone, as the lengths are on the device: where few queries
  // see many keys pairs would be up to a sixth faster (512 x 32 heads behind 16384 keys 309, 263; 2048 behind 65536
  // 2570, 2213; one prompt of 2048 without causality 100, 92).
  const bool pair = p.max_q > 2048;
  if (!(pair ? prompt_pair_layout(&a, c->num_sms, c->max_smem_optin) : prompt_mma_layout(&a, c->num_sms, c->max_smem_optin)))
    return fail(c, LI_ERR_UNSUPPORTED, "%s: operands too large for shared memory", what);
  li_status s = rows_map(c, &a.map_q, p.q, 128, p.d_nope + p.d_rope, p.H, p.total_q, p.q_head_stride, p.q_tok_stride);
  if (s == LI_OK && p.total_k > 0) {
    s = rows_map(c, &a.map_k, p.k_nope, a.box_rows, p.d_nope, p.H, p.total_k, p.k_head_stride, p.k_tok_stride);
    if (s == LI_OK) s = rows_map(c, &a.map_v, p.v, a.box_rows, p.d_v, p.H, p.total_k, p.v_head_stride, p.v_tok_stride);
    if (s == LI_OK && p.d_rope) s = rows_map(c, &a.map_kr, p.k_rope, a.box_rows, p.d_rope, 0, p.total_k, 0, p.kr_tok_stride);
  }
  if (s != LI_OK) return s;
  (void)cudaGetLastError();
  Launch L(c, st, pair ? "prompt_pair" : "prompt_attn", a.grid, pair ? 640 : 352, static_cast<int>(a.smem_bytes));
  const cudaError_t e = pair ? launch_prompt_pair(a, st) : launch_prompt_mma(a, st);
  L.done();
  return e == cudaSuccess ? LI_OK : cuda_fail(c, e, "prompt attention launch");
}

li_status prompt_attention(li_ctx* c, const li_prompt* p, void* out, float* lse, void* ws, size_t ws_bytes, cudaStream_t st) {
  const char* what = "li_prompt_attention";
  if (!p) return fail(c, LI_ERR_ARG, "%s: the argument record is NULL", what);
  li_status s = check_type(c, p->dtype, what);
  if (s != LI_OK) return s;
  if (p->H < 1 || p->batch < 1 || p->total_q < 0 || p->total_k < 0 || p->max_q < 0)
    return fail(c, LI_ERR_SHAPE, "%s: need H, batch >= 1 and total_q, total_k, max_q >= 0", what);
  const int eb = elt_bytes(p->dtype), m = 16 / eb;
  if (p->d_nope < 1 || p->d_nope > 128 || p->d_rope < 0 || p->d_rope > 64 || p->d_v < 1 || p->d_v > 128 || p->d_nope % m ||
      p->d_rope % m || p->d_v % m)
    return fail(c, LI_ERR_SHAPE, "%s: need d_nope in [1, 128], d_rope in [0, 64], d_v in [1, 128], multiples of %d", what, m);
  if (static_cast<int64_t>(p->total_q) * p->H >= (int64_t(1) << 31)) return fail(c, LI_ERR_SHAPE, "%s: total_q * H too large", what);
  if (p->H > 65535 || p->batch > 65535) return fail(c, LI_ERR_SHAPE, "%s: H and batch must be <= 65535", what);
  if (!p->cu_q || !p->cu_k) return fail(c, LI_ERR_ARG, "%s: cu_q and cu_k must be non-NULL", what);
  if (!aligned(p->cu_q, 4) || !aligned(p->cu_k, 4) || !aligned(lse, 4))
    return fail(c, LI_ERR_ALIGN, "%s: cu_q, cu_k and lse must be 4-byte aligned", what);
  if (!std::isfinite(p->scale)) return fail(c, LI_ERR_ARG, "%s: scale must be finite", what);
  if (p->total_q > 0 && (!p->q || !out)) return fail(c, LI_ERR_ARG, "%s: q and out must be non-NULL", what);
  if (p->total_k > 0 && (!p->k_nope || !p->v || (p->d_rope && !p->k_rope)))
    return fail(c, LI_ERR_ARG, "%s: k_nope, v and (with d_rope) k_rope must be non-NULL", what);
  if (!aligned(p->q, 16) || !aligned(p->k_nope, 16) || !aligned(p->k_rope, 16) || !aligned(p->v, 16) || !aligned(out, 16))
    return fail(c, LI_ERR_ALIGN, "%s: every row must be 16-byte aligned", what);
  // strides of dimensions of one element are never stepped
  const struct { int64_t stride, count; } steps[] = {
      {p->q_head_stride, p->H}, {p->k_head_stride, p->H}, {p->v_head_stride, p->H}, {p->q_tok_stride, p->total_q},
      {p->k_tok_stride, p->total_k}, {p->v_tok_stride, p->total_k}, {p->kr_tok_stride, p->d_rope ? p->total_k : 0}};
  for (const auto& d : steps)
    if (d.count > 1) {
      if (d.stride % m) return fail(c, LI_ERR_ALIGN, "%s: every row must be 16-byte aligned", what);
      if (d.stride <= 0) return fail(c, LI_ERR_ARG, "%s: strides must be positive", what);
    }
  if ((s = check_attn_ws(c, ws, ws_bytes, li_attention_workspace_bytes(c, p->H, p->d_v), what)) != LI_OK) return s;
  if ((s = check_device(c, what)) != LI_OK) return s;
  if (p->total_q == 0 || p->max_q == 0) return LI_OK;
  li_prompt a = *p;
  a.max_q = std::min(p->max_q, p->total_q);
  if (p->dtype == LI_BF16) return prompt_mma(c, a, out, lse, ws, st);
  (void)cudaGetLastError();
  Launch L(c, st, "prompt_attn_rows", 0, 256, 0);
  const cudaError_t e = launch_prompt_attn_rows(a, static_cast<float*>(out), lse, st);
  L.done();
  return e == cudaSuccess ? LI_OK : cuda_fail(c, e, "prompt attention launch");
}

}  // namespace

extern "C" {

size_t li_attention_workspace_bytes(const li_ctx* c, int H, int d_v) {
  if (!c || H < 1 || d_v < 1 || d_v > 512) return 0;
  return kAttnHeader + up256(static_cast<size_t>(c->num_sms) * sizeof(int4)) + latent_part_bytes(c->num_sms, d_v);
}

li_status li_norm_rope(li_ctx* c, const li_head_rows* sets, int n_sets, li_dtype dtype, int64_t n_tok, const int32_t* pos,
                       void* stream) try {
  if (!c) return LI_ERR_ARG;
  return norm_rope(c, sets, n_sets, dtype, n_tok, pos, static_cast<cudaStream_t>(stream));
} catch (...) {
  return LI_ERR_CUDA;
}

li_status li_append_paged(li_ctx* c, const li_paged_cache* cache, const void* x, int T, int64_t tok_stride,
                          const li_row_transform* tf, const int32_t* start, const int32_t* n_new, void* ws,
                          size_t ws_bytes, void* stream) try {
  if (!c) return LI_ERR_ARG;
  return append_paged(c, cache, x, T, tok_stride, tf, start, n_new, ws, ws_bytes, static_cast<cudaStream_t>(stream));
} catch (...) {
  return LI_ERR_CUDA;
}

li_status li_latent_attention(li_ctx* c, const li_paged_cache* cache, const void* q, int T, int H, int d_v, float scale,
                              const int32_t* q_pos, const int32_t* sel, int k, void* out, float* lse, void* ws,
                              size_t ws_bytes, void* stream) try {
  if (!c) return LI_ERR_ARG;
  return latent_attention(c, cache, q, T, H, d_v, scale, q_pos, sel, k, out, lse, ws, ws_bytes,
                          static_cast<cudaStream_t>(stream));
} catch (...) {
  return LI_ERR_CUDA;
}

li_status li_prompt_attention(li_ctx* c, const li_prompt* p, void* out, float* lse, void* ws, size_t ws_bytes,
                              void* stream) try {
  if (!c) return LI_ERR_ARG;
  return prompt_attention(c, p, out, lse, ws, ws_bytes, static_cast<cudaStream_t>(stream));
} catch (...) {
  return LI_ERR_CUDA;
}

}  // extern "C"
