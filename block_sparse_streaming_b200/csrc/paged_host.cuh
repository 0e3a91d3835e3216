// paged_host.cuh - host side of the serving and training operators around the
// attention: the page plan, the position rotation, the norm of query and key
// heads with its gradient, and the decode over paged K and V pools. Included
// by loza_ssa.cu, whose helpers (window checks, launch count) it uses.
#pragma once

#include <cmath>

namespace loza {
LOZA_NR_INSTANCES(extern, float);
LOZA_NR_INSTANCES(extern, __half);
LOZA_NR_INSTANCES(extern, __nv_bfloat16);

namespace {

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Memory of a call: `rows` rows of `len` bytes, `stride` bytes apart.
struct Extent {
  uintptr_t at;
  uint64_t len;
  uint64_t rows = 1, stride = 0;
  Extent(const void* p, uint64_t len, uint64_t rows = 1, uint64_t stride = 0)
      : at(reinterpret_cast<uintptr_t>(p)), len(len), rows(rows), stride(stride) {}
};
// Whether two share a byte; b is one row.
bool overlap(const Extent& a, const Extent& b) {
  if (a.len == 0 || a.rows == 0 || b.len == 0) return false;
  uint64_t r = 0;  // the first row of a that ends behind b's begin
  if (b.at > a.at && a.rows > 1) {
    r = (b.at - a.at) / a.stride;
    if (b.at - a.at - r * a.stride >= a.len) ++r;
  }
  return r < a.rows && a.at + r * a.stride < b.at + b.len && b.at < a.at + r * a.stride + a.len;
}

// Of a power of two.
int log2_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

// ---------------------------------------------------------------------------
// Norm and rotation
// ---------------------------------------------------------------------------
int elt_size(int dtype) { return dtype == LOZA_FP32 ? 4 : 2; }

// Shape checks that forward and backward share; fills everything but the task counts.
loza_status nr_shape(NrShape* s, int64_t tokens, int32_t d, int32_t norm_dim, float eps, const int32_t* positions,
                     const double* inv_freq, const loza_rope_params& r, int dtype) {
  if (dtype != LOZA_BF16 && dtype != LOZA_FP16 && dtype != LOZA_FP32) return LOZA_ERR_INVALID_ARG;
  if (tokens < 0 || tokens > (1 << 30) || d < 1 || norm_dim < 0 || norm_dim > d) return LOZA_ERR_INVALID_ARG;
  if (d > 1024) return LOZA_ERR_UNSUPPORTED;
  if (r.rope_dim < 0 || r.rope_dim % 2 != 0 || r.rope_offset < 0 || (int64_t)r.rope_offset + r.rope_dim > d)
    return LOZA_ERR_INVALID_ARG;
  if (r.interleaved != 0 && r.interleaved != 1) return LOZA_ERR_INVALID_ARG;
  if (!(eps >= 0.f)) return LOZA_ERR_INVALID_ARG;
  if (r.rope_dim > 0 && tokens > 0 &&
      (!positions || !inv_freq || !aligned_to(positions, 4) || !aligned_to(inv_freq, 8)))
    return LOZA_ERR_INVALID_ARG;
  *s = NrShape{};
  s->d = d;
  s->norm_dim = norm_dim;
  s->rope_off = r.rope_offset;
  s->pairs = r.rope_dim / 2;
  s->interleaved = r.interleaved;
  s->scale = r.scale;
  s->sign = 1.f;
  s->eps = eps;
  s->inv_norm = norm_dim > 0 ? 1.f / (float)norm_dim : 0.f;
  s->inv_freq = inv_freq;
  s->positions = positions;
  s->tokens = tokens;
  return LOZA_OK;
}

bool nr_rows_ok(const void* x, int64_t stride, int heads, int d, int size) {
  return x && aligned_to(x, size) && stride >= (int64_t)heads * d && stride < (int64_t(1) << 40);
}

// Largest vector (in elements) that every size, offset, stride and address
// allows: 16 bytes, for 16-bit types 4 bytes, or one element. Norm + rotation
// of 8,192 tokens with 32 + 8 heads (bf16): heads of 128 in 16-byte vectors
// took 41 us; heads of 100 in 4-byte vectors 70 us, element by element twice that.
int nr_vec(const NrShape& s, int size, std::initializer_list<const void*> ptrs, std::initializer_list<int64_t> sizes) {
  for (int v : {16 / size, 2}) {
    if (v == 2 && size == 4) continue;
    bool fits = s.d % v == 0 && s.norm_dim % v == 0 && s.rope_off % v == 0 && s.pairs % v == 0;
    for (const void* p : ptrs) fits = fits && aligned_to(p, (size_t)v * size);
    for (int64_t n : sizes) fits = fits && n % v == 0;
    if (fits) return v;
  }
  return 1;
}

// Tasks (pairs of vectors) of a row, and how many a lane takes; returns that number (NV).
int nr_tasks(NrShape* s, int vec) {
  s->nrope = s->pairs / vec;
  s->npass = (s->d - 2 * s->pairs) / vec;
  s->ntasks = s->nrope + (s->npass + 1) / 2;
  int nv = vec > 2 ? 1 : 4;
  while (nv * 32 < s->ntasks) nv = vec == 1 ? 16 : nv * 2;
  s->lph_log = 0;
  while ((nv << s->lph_log) < s->ntasks) ++s->lph_log;
  s->lph = 1 << s->lph_log;
  return nv;
}

template <typename Params>
bool nr_run(const Params& p, int dtype, int vec, int nv, int ctas, cudaStream_t st) {
  return dtype == LOZA_FP32   ? nr_run_type<float>(p, vec, nv, ctas, st)
         : dtype == LOZA_BF16 ? nr_run_type<__nv_bfloat16>(p, vec, nv, ctas, st)
                              : nr_run_type<__half>(p, vec, nv, ctas, st);
}

// Warps that fill the GPU.
int64_t nr_warps(int vec, int nv) { return (int64_t)sm_count() * nr_warps_per_sm(vec, nv); }

// Log2 of the warps that share a token: as many as find room beside each
// other on the GPU's `warps`; at most `most`, and never more than the widest
// side has groups.
int nr_wide(int64_t tokens, int64_t groups, int64_t warps, int64_t most) {
  int w = 0;
  while ((int64_t(2) << w) <= std::min(groups, most) && (tokens << (w + 1)) <= warps) ++w;
  return w;
}

// Tokens of a step of a CTA of `warps` warps, whose angles are formed together:
// four per warp (or group of warps) as far as they fit. One per warp instead of
// four: the gradient of 32,749 tokens 201 against 195 us, norm + rotation of
// 16,381 (then by CTAs of 8 warps) 78 against 75.
int nr_batch(const NrShape& s, int warps, int wide_log) {
  const int step = std::max(1, warps >> wide_log);
  int each = 4;
  while (each > 1 && (int64_t)step * each * s.pairs * (int64_t)sizeof(float2) > kNrTableBytes * warps) each /= 2;
  return step * each;
}

// The forward's walks, from the groups of the widest side and of a whole token.
// With fewer tokens than warps several warps share a walk. With many, equal
// shares end up to 40 % apart: SMs do not get equal parts of the memory's
// bandwidth (a pure copy's CTAs ended between 60 and 135 us). Short walks that
// the hardware deals out as warps end even this out, but each starts with an
// empty ring and angles to form, so a token must have groups enough, and the
// memory must be what the call waits for. Equal shares / short walks, us, of
// 16,384 tokens unless said, groups of a token in brackets:
// - One task a lane, rotation alone, from 8 groups: 64 heads of 192 (32) 152 /
//   127, 32 heads of 128 (8) 52 / 46, of 64 heads of 64 (8) 52 / 45; fewer:
//   16 heads of 128 (4) 24 / 30, 8 of 192 (4) 22 / 27, but 28 of 128 (7) 47 / 41.
// - With weights, from 12: 32 + 8 heads of 128 (12) 76 / 74, 40 + 8 (14) 92 /
//   84, 64 + 8 (20) 128 / 110, 64 + 64 of 192 (80), 8,192 tokens, 226 / 190, fp32
//   32 + 8 of 64 (12) 79 / 68; fewer: 28 + 8 of 128 (11) 70 / 71, 16 + 4 of 256
//   (11) 71 / 75, but fp32 14 + 4 of 128 (11) 74 / 67. Rows whose lanes or
//   groups are not full pay for more than they load and lose 3-6 % up to some 20
//   groups: 32 + 6 of 128 (12) 70 / 74, 32 + 8 of 192 (22) 118 / 123.
// - Several tasks a lane (8 warps an SM), 8,192 tokens. Rotation alone: 12 heads
//   of 576 (12) 44 / 39, 64 (64) 216 / 192, 8 (8) 29 / 30; every 32 pairs are
//   a turn of the warp over the angles and want a group more: 16 of 1024, all
//   rotated (16) 120 / 130, 32 (32) 207 / 194. Normed queries are bound by
//   arithmetic: 16 + 1 heads of 576 (17) 90 / 106, 64 + 1 (65) 284 / 297; with
//   few normed keys beside queries that are not, 48 + 1 (49) 172 / 153, but 24 + 1
//   (25) 85 / 86, 32 + 8 (40) 137 / 144.
// Nor with vectors of less than 16 bytes (30 / 33), nor with less than one and a
// half walks per warp that fits (1.05: 15 / 19).
void nr_plan_fwd(NrFwdParams* p, int vec, int nv, int size, int64_t groups, int64_t token_groups) {
  const int64_t warps = nr_warps(vec, nv);
  p->wide_log = nr_wide(p->s.tokens, groups, warps, 64);
  p->walks = (int)std::min(p->s.tokens, warps >> p->wide_log);
  p->batch = nr_batch(p->s, 1, p->wide_log);
  const bool norm = p->q.w || p->k.w;
  const int64_t rows = 32 >> p->s.lph_log, gq = (p->q.heads + rows - 1) / rows, gk = (p->k.heads + rows - 1) / rows;
  const bool deal = nv == 1 ? token_groups >= (norm ? 12 : 8)
                    : norm  ? !p->q.w && gq >= 8 * gk && token_groups >= 32
                            : token_groups >= 11 + p->s.pairs / 32;
  if (vec * size == 16 && p->wide_log == 0 && deal) {
    const int64_t least = norm ? 20 : 12;  // groups of a walk
    const int64_t walk = (least + token_groups - 1) / token_groups;
    const int64_t walks = (p->s.tokens + walk - 1) / walk;
    if (walks * 2 >= warps * 3) {
      p->walk = (int)walk;
      p->walks = (int)walks;
    }
  }
}

// CTAs of the backward at most (the workspace holds a row of sums per side for each).
int nr_bwd_max_ctas() { return sm_count() * 2; }

bool pool_page_ok(const loza_kv_pool& p) {
  return p.num_pages >= 1 && p.page_size >= 1 && p.page_size <= 65536 && (p.page_size & (p.page_size - 1)) == 0 &&
         (int64_t)p.num_pages * p.page_size <= INT32_MAX;
}
bool pool_strides_ok(int64_t page, int64_t row, int64_t head) {
  const int64_t cap = int64_t(1) << 40;
  return page >= 0 && row >= 0 && head >= 0 && page < cap && row < cap && head < cap;
}

// ---------------------------------------------------------------------------
// Paged K/V decode
// ---------------------------------------------------------------------------
int pkv_ctas() { return sm_count() * kPkvCtasPerSm; }

bool pkv_shape_ok(int32_t n_heads, int32_t n_kv, int32_t d_qk, int32_t d_v) {
  return n_heads >= 1 && n_kv >= 1 && n_heads % n_kv == 0 && n_kv <= 65535 && n_heads <= 65535 &&
         ((d_qk == 64 && d_v == 64) || (d_qk == 128 && d_v == 128) || (d_qk == 192 && d_v == 128));
}

size_t pkv_part_o_bytes(int32_t d_v) { return (size_t)pkv_ctas() * 2 * kPkvHeads * d_v * sizeof(float); }
size_t pkv_workspace_bytes(int32_t d_v) {
  return pkv_part_o_bytes(d_v) + (size_t)pkv_ctas() * (2 * kPkvHeads * 2 * sizeof(float) + sizeof(int4));
}

}  // namespace
}  // namespace loza

using namespace loza;

extern "C" {

loza_status loza_page_plan(const loza_page_plan_args* args, loza_stream_t stream) {
  if (!args) return LOZA_ERR_INVALID_ARG;
  const loza_page_plan_args a = *args;
  if (a.batch < 1 || a.n_free < 0 || a.max_pages < 0 || a.capacity < 0 || a.capacity > INT32_MAX)
    return LOZA_ERR_INVALID_ARG;
  if (a.page_size < 1 || a.page_size > 65536 || (a.page_size & (a.page_size - 1)) != 0) return LOZA_ERR_INVALID_ARG;
  if (!a.ctx_lens || !a.new_lens || !a.cu_seqlens || !a.seqlens || !a.counts) return LOZA_ERR_INVALID_ARG;
  if ((a.n_free > 0 && !a.free_pages) || (a.max_pages > 0 && !a.block_table) || a.bt_stride < a.max_pages)
    return LOZA_ERR_INVALID_ARG;
  if (a.capacity > 0 && (!a.positions || !a.slots || !aligned16(a.positions) || !aligned16(a.slots)))
    return LOZA_ERR_INVALID_ARG;
  for (const void* x : {(const void*)a.ctx_lens, (const void*)a.new_lens, (const void*)a.free_pages,
                        (const void*)a.block_table, (const void*)a.cu_seqlens, (const void*)a.seqlens,
                        (const void*)a.counts})
    if (!aligned_to(x, 4)) return LOZA_ERR_INVALID_ARG;
  if (a.batch > kPlanMaxBatch) return LOZA_ERR_UNSUPPORTED;
  // every CTA reads the lengths again after the first one has written seqlens: in place they would advance twice
  const uint64_t B = a.batch, cap = a.capacity;
  const Extent table(a.block_table, (uint64_t)a.max_pages * 4, B, (uint64_t)a.bt_stride * 4);
  const Extent in[] = {{a.ctx_lens, B * 4}, {a.new_lens, B * 4}, {a.free_pages, (uint64_t)a.n_free * 4}};
  const Extent out[] = {{a.cu_seqlens, (B + 1) * 4}, {a.seqlens, B * 4}, {a.counts, 12}, {a.positions, cap * 4},
                        {a.slots, cap * 8}};
  for (const Extent& x : in)
    if (overlap(table, x)) return LOZA_ERR_INVALID_ARG;
  for (const Extent& o : out) {
    if (overlap(table, o)) return LOZA_ERR_INVALID_ARG;
    for (const Extent& x : in)
      if (overlap(o, x)) return LOZA_ERR_INVALID_ARG;
    for (const Extent* x = out; x != &o; ++x)
      if (overlap(o, *x)) return LOZA_ERR_INVALID_ARG;
  }
  PlanParams p{};
  p.ctx = a.ctx_lens;
  p.add = a.new_lens;
  p.free_pages = a.free_pages;
  p.table = a.block_table;
  p.table_stride = a.bt_stride;
  p.batch = a.batch;
  p.max_pages = a.max_pages;
  p.n_free = a.n_free;
  p.page_shift = log2_of(a.page_size);
  p.capacity = a.capacity;
  p.cu = a.cu_seqlens;
  p.seqlens = a.seqlens;
  p.positions = a.positions;
  p.slots = a.slots;
  p.counts = a.counts;
  const size_t smem = (size_t)(a.batch + 1) * 2 * sizeof(int);
  // the same limit from every call: another thread's plan may be about to launch with a size of its own
  constexpr size_t most = (size_t)(kPlanMaxBatch + 1) * 2 * sizeof(int);
  if (smem > 48 * 1024 && cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)most) != cudaSuccess)
    return LOZA_ERR_CUDA;
  // four tokens a thread; new pages are at most one a request more than tokens / page_size
  const int64_t work = std::max<int64_t>((a.capacity + 3) / 4, a.batch);
  const unsigned grid = (unsigned)std::max<int64_t>(
      1, std::min<int64_t>((work + kPlanThreads - 1) / kPlanThreads, (int64_t)sm_count() * 2));
  page_plan_kernel<<<grid, kPlanThreads, smem, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return cudaGetLastError() == cudaSuccess ? LOZA_OK : LOZA_ERR_CUDA;
}

loza_status loza_rope_frequencies(double theta, int32_t rope_dim, int32_t scaling, double factor, double original_max,
                                  double beta_fast, double beta_slow, double* inv_freq, float* scale) {
  if (rope_dim < 2 || rope_dim % 2 != 0 || rope_dim > 1024 || !inv_freq || !scale) return LOZA_ERR_INVALID_ARG;
  if (!(theta > 1.0) || !std::isfinite(theta) || !(factor >= 1.0) || !std::isfinite(factor))
    return LOZA_ERR_INVALID_ARG;
  const int half = rope_dim / 2;
  const double pi2 = 6.28318530717958647693;
  *scale = 1.f;
  if (scaling == LOZA_ROPE_NTK) {
    if (rope_dim == 2) return LOZA_ERR_INVALID_ARG;  // its exponent dim / (dim - 2)
    theta *= std::pow(factor, (double)rope_dim / (rope_dim - 2));
  }
  double low = 0, high = 0;
  if (scaling == LOZA_ROPE_YARN) {
    if (!(original_max >= 1.0) || !(beta_slow > 0.0) || !(beta_fast > beta_slow)) return LOZA_ERR_INVALID_ARG;
    // the (fractional) pair index whose frequency makes `turns` turns over the original length, times two
    auto column = [&](double turns) {
      return rope_dim * std::log(original_max / (turns * pi2)) / (2 * std::log(theta));
    };
    low = std::max(std::floor(column(beta_fast)), 0.0);
    high = std::min(std::ceil(column(beta_slow)), (double)rope_dim - 1);
    *scale = factor > 1.0 ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
  } else if (scaling != LOZA_ROPE_NONE && scaling != LOZA_ROPE_LINEAR && scaling != LOZA_ROPE_NTK) {
    return LOZA_ERR_INVALID_ARG;
  }
  for (int i = 0; i < half; ++i) {
    double f = std::pow(theta, -(double)i / half);
    if (scaling == LOZA_ROPE_LINEAR) f /= factor;
    if (scaling == LOZA_ROPE_YARN) {
      const double ramp = std::min(1.0, std::max(0.0, (i - low) / std::max(high - low, 0.001)));
      f = f / factor * ramp + f * (1.0 - ramp);
    }
    inv_freq[i] = f;
  }
  return LOZA_OK;
}

loza_status loza_rope(const loza_rope_args* args, loza_stream_t stream) {
  if (!args) return LOZA_ERR_INVALID_ARG;
  const loza_rope_args a = *args;
  NrFwdParams p{};
  const loza_status rc = nr_shape(&p.s, a.tokens, a.d, 0, 0.f, a.positions, a.inv_freq, a.rope, a.dtype);
  if (rc != LOZA_OK) return rc;
  if (a.n_heads < 1 || a.n_heads > 65535 || (a.transposed != 0 && a.transposed != 1)) return LOZA_ERR_INVALID_ARG;
  if (a.tokens == 0) return LOZA_OK;
  const int size = elt_size(a.dtype);
  if (!nr_rows_ok(a.x, a.x_row_stride, a.n_heads, a.d, size) ||
      !nr_rows_ok(a.out, a.out_row_stride, a.n_heads, a.d, size))
    return LOZA_ERR_INVALID_ARG;
  if (a.x == a.out && a.x_row_stride != a.out_row_stride) return LOZA_ERR_INVALID_ARG;
  if (a.x == a.out && a.rope.rope_dim == 0) return LOZA_OK;
  if (a.transposed) p.s.sign = -1.f;
  p.q.x = a.x;
  p.q.x_stride = a.x_row_stride;
  p.q.out = a.out;
  p.q.out_stride = a.out_row_stride;
  p.q.heads = a.n_heads;
  const int vec = nr_vec(p.s, size, {a.x, a.out}, {a.x_row_stride, a.out_row_stride});
  int nv = nr_tasks(&p.s, vec);
  if (a.x == a.out) {  // in place: the rotated columns alone
    p.s.npass = 0;
    p.s.ntasks = p.s.nrope;
    p.s.lph_log = 0;
    while ((nv << p.s.lph_log) < p.s.ntasks) ++p.s.lph_log;
    p.s.lph = 1 << p.s.lph_log;
  }
  const int rows = 32 >> p.s.lph_log;
  const int64_t groups = (a.n_heads + rows - 1) / rows;
  nr_plan_fwd(&p, vec, nv, size, groups, groups);
  if (!nr_run(p, a.dtype, vec, nv, 0, reinterpret_cast<cudaStream_t>(stream))) return LOZA_ERR_CUDA;
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return LOZA_OK;
}

loza_status loza_qk_norm_rope(const loza_qk_norm_rope_args* args, loza_stream_t stream) {
  if (!args) return LOZA_ERR_INVALID_ARG;
  const loza_qk_norm_rope_args a = *args;
  const loza_kv_pool* pool = a.pool.k ? &a.pool : nullptr;
  NrFwdParams p{};
  const loza_status rc = nr_shape(&p.s, a.tokens, a.d, a.norm_dim, a.eps, a.positions, a.inv_freq, a.rope, a.dtype);
  if (rc != LOZA_OK) return rc;
  if (a.n_heads < 0 || a.n_kv_heads < 0 || a.n_heads > 65535 || a.n_kv_heads > 65535 || a.n_heads + a.n_kv_heads < 1)
    return LOZA_ERR_INVALID_ARG;
  const int size = elt_size(a.dtype);
  if ((a.q_weight || a.k_weight) && a.norm_dim < 1) return LOZA_ERR_INVALID_ARG;
  if (!aligned_to(a.q_weight, size) || !aligned_to(a.k_weight, size)) return LOZA_ERR_INVALID_ARG;
  if (pool) {
    if (!pool_page_ok(*pool) || !aligned_to(pool->k, size) ||
        !pool_strides_ok(pool->k_page_stride, pool->k_row_stride, pool->k_head_stride))
      return LOZA_ERR_INVALID_ARG;
    if (a.n_kv_heads < 1 || (a.tokens > 0 && (!a.slots || !aligned_to(a.slots, 8)))) return LOZA_ERR_INVALID_ARG;
    if ((a.v != nullptr) != (pool->v != nullptr)) return LOZA_ERR_INVALID_ARG;
    if (a.v && (a.d_v < 1 || a.d_v > 1024 || !aligned_to(pool->v, size) ||
                !pool_strides_ok(pool->v_page_stride, pool->v_row_stride, pool->v_head_stride)))
      return LOZA_ERR_INVALID_ARG;
  } else if (a.v || a.slots) {
    return LOZA_ERR_INVALID_ARG;  // values and slots are for the pool
  }
  if (a.n_kv_heads > 0 && !pool && !a.k_out) return LOZA_ERR_INVALID_ARG;
  if (a.tokens == 0) return LOZA_OK;
  if (a.n_heads > 0 && (!nr_rows_ok(a.q, a.q_row_stride, a.n_heads, a.d, size) ||
                        !nr_rows_ok(a.q_out, a.q_out_row_stride, a.n_heads, a.d, size)))
    return LOZA_ERR_INVALID_ARG;
  if (a.n_kv_heads > 0 && (!nr_rows_ok(a.k, a.k_row_stride, a.n_kv_heads, a.d, size) ||
                           (a.k_out && !nr_rows_ok(a.k_out, a.k_out_row_stride, a.n_kv_heads, a.d, size))))
    return LOZA_ERR_INVALID_ARG;
  if (a.v && !nr_rows_ok(a.v, a.v_row_stride, a.n_kv_heads, a.d_v, size)) return LOZA_ERR_INVALID_ARG;
  if ((a.n_heads > 0 && a.q == a.q_out && a.q_row_stride != a.q_out_row_stride) ||
      (a.n_kv_heads > 0 && a.k == a.k_out && a.k_row_stride != a.k_out_row_stride))
    return LOZA_ERR_INVALID_ARG;
  if (a.n_heads > 0) {
    p.q = NrSide{a.q, nullptr, a.q_weight, a.q_out, a.q_row_stride, 0, a.q_out_row_stride, a.n_heads,
                 a.q == a.q_out && !a.q_weight};
  }
  if (a.n_kv_heads > 0) {
    p.k = NrSide{a.k, nullptr, a.k_weight, a.k_out, a.k_row_stride, 0, a.k_out ? a.k_out_row_stride : 0, a.n_kv_heads,
                 a.k == a.k_out && !a.k_weight && !pool};
  }
  if (pool) {
    p.k_pool = NrPool{pool->k, pool->k_page_stride, pool->k_row_stride, pool->k_head_stride};
    if (a.v) p.v_pool = NrPool{pool->v, pool->v_page_stride, pool->v_row_stride, pool->v_head_stride};
    p.page_shift = log2_of(pool->page_size);
    p.n_slots = (int64_t)pool->num_pages * pool->page_size;
    p.slots = a.slots;
  }
  p.v = a.v;
  p.v_stride = a.v_row_stride;
  p.d_v = a.v ? a.d_v : 0;
  // arguments that are not given are null or zero here and constrain nothing
  const int vec = nr_vec(p.s, size,
                         {p.q.x, p.q.out, p.q.w, p.k.x, p.k.out, p.k.w, p.k_pool.base, p.v_pool.base, p.v},
                         {p.q.x_stride, p.q.out_stride, p.k.x_stride, p.k.out_stride, p.k_pool.page_stride,
                          p.k_pool.row_stride, p.k_pool.head_stride, p.v_pool.page_stride, p.v_pool.row_stride,
                          p.v_pool.head_stride, a.v ? p.v_stride : 0, p.d_v});
  const int nv = nr_tasks(&p.s, vec);
  const int rows = 32 >> p.s.lph_log;
  const int vper = p.d_v / vec;
  p.vper_log = vper > 0 && (vper & (vper - 1)) == 0 ? log2_of(vper) : -1;
  const int64_t gq = (a.n_heads + rows - 1) / rows, gk = (a.n_kv_heads + rows - 1) / rows;
  nr_plan_fwd(&p, vec, nv, size, std::max(gq, gk), gq + gk + ((int64_t)a.n_kv_heads * vper + 63) / 64);
  if (!nr_run(p, a.dtype, vec, nv, 0, reinterpret_cast<cudaStream_t>(stream))) return LOZA_ERR_CUDA;
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return LOZA_OK;
}

size_t loza_qk_norm_rope_workspace_size(int32_t norm_dim) {
  if (norm_dim < 1 || norm_dim > 1024) return 0;
  return (size_t)2 * nr_bwd_max_ctas() * norm_dim * sizeof(float);
}

loza_status loza_qk_norm_rope_backward(const loza_qk_norm_rope_backward_args* args, loza_stream_t stream) {
  if (!args) return LOZA_ERR_INVALID_ARG;
  const loza_qk_norm_rope_backward_args a = *args;
  NrBwdParams p{};
  const loza_status rc = nr_shape(&p.s, a.tokens, a.d, a.norm_dim, a.eps, a.positions, a.inv_freq, a.rope, a.dtype);
  if (rc != LOZA_OK) return rc;
  if (a.n_heads < 0 || a.n_kv_heads < 0 || a.n_heads > 65535 || a.n_kv_heads > 65535 || a.n_heads + a.n_kv_heads < 1)
    return LOZA_ERR_INVALID_ARG;
  const int size = elt_size(a.dtype);
  if ((a.q_weight || a.k_weight) && a.norm_dim < 1) return LOZA_ERR_INVALID_ARG;
  if ((a.q_weight && a.n_heads < 1) || (a.k_weight && a.n_kv_heads < 1)) return LOZA_ERR_INVALID_ARG;
  if (!aligned_to(a.q_weight, size) || !aligned_to(a.k_weight, size)) return LOZA_ERR_INVALID_ARG;
  if ((a.q_weight != nullptr) != (a.dq_weight != nullptr) || (a.k_weight != nullptr) != (a.dk_weight != nullptr))
    return LOZA_ERR_INVALID_ARG;
  if (!aligned_to(a.dq_weight, 4) || !aligned_to(a.dk_weight, 4)) return LOZA_ERR_INVALID_ARG;
  if (a.dq_weight && a.dk_weight &&
      overlap({a.dq_weight, (uint64_t)a.norm_dim * 4}, {a.dk_weight, (uint64_t)a.norm_dim * 4}))
    return LOZA_ERR_INVALID_ARG;  // a weight of both sides has two gradients, which the caller adds
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (a.tokens == 0) {  // the weights' gradients are sums over nothing
    if (a.dq_weight && cudaMemsetAsync(a.dq_weight, 0, (size_t)a.norm_dim * 4, st) != cudaSuccess) return LOZA_ERR_CUDA;
    if (a.dk_weight && cudaMemsetAsync(a.dk_weight, 0, (size_t)a.norm_dim * 4, st) != cudaSuccess) return LOZA_ERR_CUDA;
    return LOZA_OK;
  }
  if (a.n_heads > 0 && (!nr_rows_ok(a.dq_out, a.dq_out_row_stride, a.n_heads, a.d, size) ||
                        !nr_rows_ok(a.dq, a.dq_row_stride, a.n_heads, a.d, size) ||
                        (a.q_weight && !nr_rows_ok(a.q, a.q_row_stride, a.n_heads, a.d, size))))
    return LOZA_ERR_INVALID_ARG;
  if (a.n_kv_heads > 0 && (!nr_rows_ok(a.dk_out, a.dk_out_row_stride, a.n_kv_heads, a.d, size) ||
                           !nr_rows_ok(a.dk, a.dk_row_stride, a.n_kv_heads, a.d, size) ||
                           (a.k_weight && !nr_rows_ok(a.k, a.k_row_stride, a.n_kv_heads, a.d, size))))
    return LOZA_ERR_INVALID_ARG;
  // a gradient may replace its own input (the same rows), nothing else
  if ((a.n_heads > 0 && ((a.dq == a.dq_out && a.dq_row_stride != a.dq_out_row_stride) ||
                         (a.q_weight && a.dq == a.q && a.dq_row_stride != a.q_row_stride))) ||
      (a.n_kv_heads > 0 && ((a.dk == a.dk_out && a.dk_row_stride != a.dk_out_row_stride) ||
                            (a.k_weight && a.dk == a.k && a.dk_row_stride != a.k_row_stride))))
    return LOZA_ERR_INVALID_ARG;
  const bool sums = a.q_weight || a.k_weight;
  if (sums) {
    if (!a.workspace || !aligned16(a.workspace)) return LOZA_ERR_INVALID_ARG;
    if (a.workspace_bytes < loza_qk_norm_rope_workspace_size(a.norm_dim)) return LOZA_ERR_WORKSPACE;
  }
  p.s.sign = -1.f;
  if (a.n_heads > 0)
    p.q = NrSide{a.q_weight ? a.q : nullptr, a.dq_out, a.q_weight, a.dq, a.q_weight ? a.q_row_stride : 0,
                 a.dq_out_row_stride, a.dq_row_stride, a.n_heads, 0};
  if (a.n_kv_heads > 0)
    p.k = NrSide{a.k_weight ? a.k : nullptr, a.dk_out, a.k_weight, a.dk, a.k_weight ? a.k_row_stride : 0,
                 a.dk_out_row_stride, a.dk_row_stride, a.n_kv_heads, 0};
  p.partial = static_cast<float*>(a.workspace);
  const int vec = nr_vec(p.s, size, {p.q.x, p.q.dy, p.q.w, p.q.out, p.k.x, p.k.dy, p.k.w, p.k.out},
                         {p.q.x_stride, p.q.dy_stride, p.q.out_stride, p.k.x_stride, p.k.dy_stride, p.k.out_stride});
  const int nv = nr_tasks(&p.s, vec);
  const int rows = 32 >> p.s.lph_log;
  const int64_t gq = (a.n_heads + rows - 1) / rows, gk = (a.n_kv_heads + rows - 1) / rows;
  const int64_t full = nr_warps(vec, nv) / kNrWarps;
  p.wide_log = nr_wide(a.tokens, std::max(gq, gk), full * kNrWarps, kNrWarps);
  const int64_t ctas = std::min(full, ((a.tokens << p.wide_log) + kNrWarps - 1) / kNrWarps);
  p.batch = nr_batch(p.s, kNrWarps, p.wide_log);
  if (!nr_run(p, a.dtype, vec, nv, (int)ctas, st)) return LOZA_ERR_CUDA;
  g_launches.fetch_add(1, std::memory_order_relaxed);
  if (sums) {
    const NrDwParams dw{p.partial, a.dq_weight, a.dk_weight, a.norm_dim, (int)ctas};
    if (!launch_after(norm_rope_dw_kernel, dim3((a.norm_dim + 7) / 8, 2), 512, st, dw)) return LOZA_ERR_CUDA;
    g_launches.fetch_add(1, std::memory_order_relaxed);
  }
  return LOZA_OK;
}

size_t loza_decode_paged_kv_workspace_size(int32_t n_heads, int32_t n_kv_heads, int32_t d_qk, int32_t d_v) {
  if (!pkv_shape_ok(n_heads, n_kv_heads, d_qk, d_v)) return 0;
  return pkv_workspace_bytes(d_v);
}

loza_status loza_ssa_decode_paged_kv(const loza_decode_paged_kv_args* args, loza_stream_t stream) {
  if (!args) return LOZA_ERR_INVALID_ARG;
  const loza_decode_paged_kv_args a = *args;
  const loza_kv_pool* pool = &a.pool;
  if (!a.q || !pool->k || !pool->v || !a.block_table || !a.seqlens || !a.out || !a.lse) return LOZA_ERR_INVALID_ARG;
  if (!aligned16(a.q) || !aligned16(pool->k) || !aligned16(pool->v) || !aligned16(a.out)) return LOZA_ERR_INVALID_ARG;
  if (!aligned_to(a.block_table, 4) || !aligned_to(a.seqlens, 4) || !aligned_to(a.lse, 4)) return LOZA_ERR_INVALID_ARG;
  if (a.batch < 1 || a.batch > 65535 || a.max_seqlen < 1 || a.max_seqlen > (1 << 30)) return LOZA_ERR_INVALID_ARG;
  if (!pool_page_ok(*pool)) return LOZA_ERR_INVALID_ARG;
  if (!pool_strides_ok(pool->k_page_stride, pool->k_row_stride, pool->k_head_stride) ||
      !pool_strides_ok(pool->v_page_stride, pool->v_row_stride, pool->v_head_stride))
    return LOZA_ERR_INVALID_ARG;
  for (int64_t s : {pool->k_page_stride, pool->k_row_stride, pool->k_head_stride, pool->v_page_stride,
                    pool->v_row_stride, pool->v_head_stride, a.q_row_stride})
    if (s % 8 != 0) return LOZA_ERR_INVALID_ARG;
  if (a.n_heads < 1 || a.n_kv_heads < 1 || a.n_heads % a.n_kv_heads != 0 || a.n_heads > 65535)
    return LOZA_ERR_INVALID_ARG;
  if (a.q_row_stride < (int64_t)a.n_heads * a.d_qk || a.q_row_stride >= (int64_t(1) << 40)) return LOZA_ERR_INVALID_ARG;
  if (a.bt_stride < ((int64_t)a.max_seqlen + pool->page_size - 1) / pool->page_size) return LOZA_ERR_INVALID_ARG;
  if (a.dtype != LOZA_BF16 && a.dtype != LOZA_FP16 && a.dtype != LOZA_FP32) return LOZA_ERR_INVALID_ARG;
  if (!window_ok(a.window) || a.dtype == LOZA_FP32 || pool->page_size < 16 ||
      !pkv_shape_ok(a.n_heads, a.n_kv_heads, a.d_qk, a.d_v))
    return LOZA_ERR_UNSUPPORTED;
  if (!a.workspace || !aligned16(a.workspace)) return LOZA_ERR_INVALID_ARG;
  if (a.workspace_bytes < pkv_workspace_bytes(a.d_v)) return LOZA_ERR_WORKSPACE;
  PagedKvParams p{};
  p.q = a.q;
  p.q_stride = a.q_row_stride;
  p.k = pool->k;
  p.v = pool->v;
  p.k_page = pool->k_page_stride;
  p.k_row = pool->k_row_stride;
  p.k_head = pool->k_head_stride;
  p.v_page = pool->v_page_stride;
  p.v_row = pool->v_row_stride;
  p.v_head = pool->v_head_stride;
  p.table = a.block_table;
  p.table_stride = a.bt_stride;
  p.seqlens = a.seqlens;
  p.batch = a.batch;
  p.max_seqlen = a.max_seqlen;
  p.num_pages = pool->num_pages;
  p.page_shift = log2_of(pool->page_size);
  p.n_kv = a.n_kv_heads;
  p.group = a.n_heads / a.n_kv_heads;
  p.chunks = (p.group + kPkvHeads - 1) / kPkvHeads;
  p.chunk = (p.group + p.chunks - 1) / p.chunks;
  p.win = host_window(a.window);
  p.scale_log2 = a.window.scale * 1.4426950408889634f;
  p.out = a.out;
  p.lse = a.lse;
  p.part_o = static_cast<float*>(a.workspace);
  p.part_ml = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + pkv_part_o_bytes(a.d_v));
  p.ctas = pkv_ctas();
  p.split = reinterpret_cast<int4*>(p.part_ml + (size_t)p.ctas * 2 * kPkvHeads * 2);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!(a.dtype == LOZA_BF16 ? pkv_run<__nv_bfloat16> : pkv_run<__half>)(p, a.d_qk, st)) return LOZA_ERR_CUDA;
  g_launches.fetch_add(2, std::memory_order_relaxed);
  return LOZA_OK;
}

}  // extern "C"
