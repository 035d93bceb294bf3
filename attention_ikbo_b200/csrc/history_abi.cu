// history_abi.cu -- host side of the history-cache entry points: argument checks and launches.
#include <cmath>
#include <cstring>

#include "history.h"

namespace rocs {
int sm_count_ext();
int check_csr_ext(const int32_t* off, int64_t R, int64_t* total);
void set_last_launches(int n);
bool tmap_bf16_3d_ext(CUtensorMap* tm, const void* base, uint64_t inner, uint64_t outer1, uint64_t outer2, uint64_t row_bytes,
                      uint64_t plane_bytes, uint32_t box_in, uint32_t box_1, uint32_t box_2);
}  // namespace rocs

using namespace rocs;

namespace {

inline bool al(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int rope_validate(const float* rope, int64_t max_pos, int64_t rot, int64_t dh) {
  if (!rope) return ROCS_OK;
  if (!al(rope, 16) || max_pos <= 0) return ROCS_ERR_INVALID_ARG;
  if (rot <= 0 || rot > dh || rot % 16 || max_pos >= (int64_t(1) << 31)) return ROCS_ERR_UNSUPPORTED;
  return ROCS_OK;
}

int workspace_validate(const void* ws, size_t have, size_t need) {
  return !ws || have < need || !al(ws, 256) ? ROCS_ERR_WORKSPACE : ROCS_OK;
}

// first and one past the last byte of n rows of `row` elements, ld elements apart
struct Span {
  uintptr_t lo, hi;
};
Span span(const void* p, int64_t n, int64_t row, int64_t ld, int64_t es) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(p);
  return {b, b + (uintptr_t)(((n - 1) * ld + row) * es)};
}
inline bool apart(const Span& a, const Span& b) { return a.hi <= b.lo || b.hi <= a.lo; }
// the same for rows of row_a and row_b bytes: also where they lie side by side in one wider buffer, ld bytes a row
bool rows_apart(const Span& a, int64_t row_a, int64_t ld_a, const Span& b, int64_t row_b, int64_t ld_b) {
  if (apart(a, b)) return true;
  if (ld_a != ld_b) return false;
  const int64_t d = (int64_t)(b.lo > a.lo ? b.lo - a.lo : a.lo - b.lo) % ld_a;
  const int64_t first = b.lo > a.lo ? row_a : row_b, second = b.lo > a.lo ? row_b : row_a;
  return d >= first && d + second <= ld_a;
}

int side_validate(const rocs_norm_rope_side& s, const rocs_norm_rope_args* a) {
  if (s.n < 0 || s.heads < 0) return ROCS_ERR_INVALID_ARG;
  if (s.n == 0) return ROCS_OK;
  if (s.heads == 0 || !s.x || !s.out) return ROCS_ERR_INVALID_ARG;
  const int64_t row = s.heads * a->dh, es = a->dtype == ROCS_BF16 ? 2 : 4;
  if (s.n >= (int64_t(1) << 31) || row >= (int64_t(1) << 24) || s.n * s.heads >= (int64_t(1) << 31)) return ROCS_ERR_UNSUPPORTED;
  const int64_t ldx = s.ld_x ? s.ld_x : row, ldo = s.ld_out ? s.ld_out : row;
  if (ldx < row || ldo < row) return ROCS_ERR_INVALID_ARG;
  if ((ldx * es) % 16 || (ldo * es) % 16 || ldx >= (int64_t(1) << 31) || ldo >= (int64_t(1) << 31)) return ROCS_ERR_UNSUPPORTED;
  if (!al(s.x, 16) || !al(s.out, 16)) return ROCS_ERR_INVALID_ARG;
  if (a->rope && (!s.pos || !al(s.pos, 4))) return ROCS_ERR_INVALID_ARG;
  if ((s.gamma && !al(s.gamma, 16)) || (s.beta && !al(s.beta, 16))) return ROCS_ERR_INVALID_ARG;
  return ROCS_OK;
}

// an output may be its own side's input in place; nothing else may overlap an output
int overlap_validate(const rocs_norm_rope_args* a) {
  const rocs_norm_rope_side* s[2] = {&a->q, &a->k};
  const int64_t es = a->dtype == ROCS_BF16 ? 2 : 4;
  for (int o = 0; o < 2; ++o) {
    if (s[o]->n == 0) continue;
    const int64_t row = s[o]->heads * a->dh, ldo = s[o]->ld_out ? s[o]->ld_out : row;
    const Span out = span(s[o]->out, s[o]->n, row, ldo, es);
    for (int i = 0; i < 4; ++i) {  // 0, 1: inputs; 2, 3: outputs
      const rocs_norm_rope_side* t = s[i & 1];
      if (t->n == 0 || (i >= 2 && (i & 1) == o)) continue;
      const int64_t rowt = t->heads * a->dh, ldt = (i < 2 ? t->ld_x : t->ld_out) ? (i < 2 ? t->ld_x : t->ld_out) : rowt;
      const void* pt = i < 2 ? t->x : t->out;
      if (i < 2 && (i & 1) == o && pt == s[o]->out && ldt == ldo) continue;
      if (rows_apart(out, row * es, ldo * es, span(pt, t->n, rowt, ldt, es), rowt * es, ldt * es)) continue;
      return ROCS_ERR_INVALID_ARG;
    }
  }
  return ROCS_OK;
}

int norm_rope_validate(const rocs_norm_rope_args* a) {
  if (!a || a->dh <= 0) return ROCS_ERR_INVALID_ARG;
  if (a->dtype != ROCS_F32 && a->dtype != ROCS_BF16) return ROCS_ERR_INVALID_ARG;
  if (a->norm < ROCS_NORM_NONE || a->norm > ROCS_NORM_RMS) return ROCS_ERR_INVALID_ARG;
  if (!(a->eps >= 0.0f) || !std::isfinite(a->eps)) return ROCS_ERR_INVALID_ARG;
  if (a->dh != 64 && a->dh != 128) return ROCS_ERR_UNSUPPORTED;
  int rc = rope_validate(a->rope, a->max_pos, a->rot, a->dh);
  if (rc || (rc = side_validate(a->q, a)) || (rc = side_validate(a->k, a))) return rc;
  return overlap_validate(a);
}

int cache_validate(const rocs_cache_q4& c) {
  if (c.pages < 0 || c.page <= 0 || c.heads <= 0 || c.dh <= 0) return ROCS_ERR_INVALID_ARG;
  if (c.dh != 64 && c.dh != 128) return ROCS_ERR_UNSUPPORTED;
  if (c.page != 16 && c.page != 32 && c.page != 64 && c.page != 128) return ROCS_ERR_UNSUPPORTED;
  if (c.pages >= (int64_t(1) << 31) || c.heads >= (int64_t(1) << 16) || c.pages * c.heads * c.page >= (int64_t(1) << 40))
    return ROCS_ERR_UNSUPPORTED;
  const void* ptrs[] = {c.k_codes, c.v_codes, c.k_scale, c.v_scale};
  for (const void* p : ptrs)
    if ((c.pages > 0 && !p) || !al(p, 16)) return ROCS_ERR_INVALID_ARG;
  return ROCS_OK;
}
// the cache's four buffers
void cache_spans(const rocs_cache_q4& c, Span (&s)[4]) {
  const int64_t rows = c.pages * c.heads * c.page;
  s[0] = span(c.k_codes, 1, rows, rows, c.dh / 2);
  s[1] = span(c.v_codes, 1, rows, rows, c.dh / 2);
  s[2] = span(c.k_scale, 1, rows, rows, 4);
  s[3] = span(c.v_scale, 1, rows, rows, 4);
}
CacheQ4 cache_of(const rocs_cache_q4& c) {
  CacheQ4 q;
  q.codes[0] = static_cast<uint8_t*>(c.k_codes);
  q.codes[1] = static_cast<uint8_t*>(c.v_codes);
  q.scale[0] = static_cast<__nv_bfloat162*>(c.k_scale);
  q.scale[1] = static_cast<__nv_bfloat162*>(c.v_scale);
  q.pages = (int)c.pages;
  q.heads = (int)c.heads;
  q.page_log2 = c.page == 16 ? 4 : c.page == 32 ? 5 : c.page == 64 ? 6 : 7;
  return q;
}

int move_validate(const rocs_cache_move_args* a, bool append, int64_t* T) {
  if (!a) return ROCS_ERR_INVALID_ARG;
  int rc = cache_validate(a->cache);
  if (rc) return rc;
  if (a->R < 0 || a->max_pages < 0) return ROCS_ERR_INVALID_ARG;
  if (a->R >= (int64_t(1) << 28) || a->max_pages >= (int64_t(1) << 27)) return ROCS_ERR_UNSUPPORTED;
  if (a->dtype != ROCS_F32 && a->dtype != ROCS_BF16) return ROCS_ERR_INVALID_ARG;
  if (!append && a->dtype != ROCS_BF16) return ROCS_ERR_UNSUPPORTED;
  if ((rc = check_csr_ext(a->tok_off_host, a->R, T))) return rc;
  if (*T == 0) return ROCS_OK;
  if (!a->tok_off_dev || !a->base || !a->k || !a->v || (a->max_pages > 0 && !a->page_table)) return ROCS_ERR_INVALID_ARG;
  if (!al(a->k, 16) || !al(a->v, 16) || !al(a->base, 4) || !al(a->page_table, 4) || !al(a->pos, 4)) return ROCS_ERR_INVALID_ARG;
  if (*T * a->cache.heads >= (int64_t(1) << 31)) return ROCS_ERR_UNSUPPORTED;
  const int64_t row = a->cache.heads * a->cache.dh, es = a->dtype == ROCS_BF16 ? 2 : 4;
  for (int64_t ld : {a->k_ld, a->v_ld}) {
    if (ld != 0 && ld < row) return ROCS_ERR_INVALID_ARG;
    if ((ld * es) % 16 || ld >= (int64_t(1) << 31)) return ROCS_ERR_UNSUPPORTED;
  }
  return append ? rope_validate(a->rope, a->max_pos, a->rot, a->cache.dh) : ROCS_OK;
}

// What a call writes must not overlap what it reads or writes elsewhere: append the cache's buffers, read k and v.
int move_overlap_validate(const rocs_cache_move_args* a, bool append, int64_t T) {
  if (T == 0) return ROCS_OK;
  const int64_t row = a->cache.heads * a->cache.dh, es = a->dtype == ROCS_BF16 ? 2 : 4;
  const int64_t ld[2] = {a->k_ld ? a->k_ld : row, a->v_ld ? a->v_ld : row};
  const Span x[2] = {span(a->k, T, row, ld[0], es), span(a->v, T, row, ld[1], es)};
  Span c[4];
  cache_spans(a->cache, c);
  for (int i = 0; i < 4; ++i) {
    if (!apart(x[0], c[i]) || !apart(x[1], c[i])) return ROCS_ERR_INVALID_ARG;
    for (int j = 0; j < i && append; ++j)
      if (!apart(c[i], c[j])) return ROCS_ERR_INVALID_ARG;
  }
  return append || rows_apart(x[0], row * es, ld[0] * es, x[1], row * es, ld[1] * es) ? ROCS_OK : ROCS_ERR_INVALID_ARG;
}

int cache_move(const rocs_cache_move_args* a, bool append, cudaStream_t st) {
  int64_t T = 0;
  int rc = move_validate(a, append, &T);
  if (rc || (rc = workspace_validate(a->workspace, a->workspace_bytes, sizeof(WsHeader))) || (rc = move_overlap_validate(a, append, T)))
    return rc;
  CacheMoveParams p;
  std::memset(&p, 0, sizeof(p));
  p.c = cache_of(a->cache);
  const int64_t row = a->cache.heads * a->cache.dh;
  p.x[0] = const_cast<void*>(a->k);
  p.x[1] = const_cast<void*>(a->v);
  p.ld[0] = a->k_ld ? a->k_ld : row;
  p.ld[1] = a->v_ld ? a->v_ld : row;
  p.tok_off = a->tok_off_dev;
  p.base = a->base;
  p.table = a->page_table;
  p.pos = a->pos;
  p.rope = append ? a->rope : nullptr;
  p.R = (int)a->R;
  p.max_pages = (int)a->max_pages;
  p.max_pos = (int)a->max_pos;
  p.rot = (int)a->rot;
  p.interleaved = a->interleaved != 0;
  p.ws = static_cast<WsHeader*>(a->workspace);
  p.rows = T * a->cache.heads;
  const int unroll = unroll_for(p.rows, a->cache.dh, sm_count_ext(), append ? kAppendSets : kReadSets);
  const int per = unroll * rows_per_warp(a->cache.dh);
  p.warps = (p.rows + per - 1) / per;
  if (cudaMemsetAsync(p.ws, 0, sizeof(WsHeader), st) != cudaSuccess) return ROCS_ERR_CUDA;
  if (T > 0) {
    const cudaError_t e = append ? launch_cache_append(p, (int)a->cache.dh, a->dtype == ROCS_F32, unroll, st)
                                 : launch_cache_read(p, (int)a->cache.dh, unroll, st);
    if (e != cudaSuccess) return ROCS_ERR_CUDA;
  }
  set_last_launches(T > 0 ? 1 : 0);
  return ROCS_OK;
}

// ---------------------------------------------------------------- attention over the cache
// Which kernel takes which request is chosen by what their units cost, as measured with equal histories (32 of 4096 keys, 8
// heads): the kernel for few rows takes 66 us (dh = 64: 41) for every 16 rows of the key heads, the one for many 150 (134)
// for up to 128 and 183 (149) for 256, so up to 32 (48) rows are about as well off with the first.  At that border the two
// took 156 and 150 us (141 and 134); with 8 histories of 16384 keys 154 and 143 (139 and 120), with 256 of 512 keys 191 and
// 182 (182 and 157).  Calls of a single kind get one kernel; calls with
// both kinds get both kernels, one after the other, only where that saves a fifth, because each ends in a tail of its own
// (16 requests of 16-64 rows of 64: 35 us with the first alone, 46 with the second alone, 62 with both).
constexpr int kFewCost = 10, kManyCost128 = 24, kManyCost64 = 34;
constexpr int kFewLimit128 = 32, kFewLimit64 = 48;
constexpr int kMaxShared = 64;  // query heads to a key head up to which a 128-row tile is well filled
inline size_t a256(size_t n) { return (n + 255) & ~size_t(255); }

// What a call needs: which kernels run (by the rows of a key head that the requests have), and the workspace
// [WsHeader][counters][partial results], the first two zeroed before every call.
struct AttnPlan {
  int64_t C = 0;
  int rows_hi = 0;  // requests with up to this many rows go to the kernel for few rows
  int rows_few = 0;  // the most that a request of the kernel for few rows has
  int grid_few = 0, grid_many = 0;  // 0: not launched
  size_t cnt_many = 0, zero = 0, bytes = 0;
};

int attn_validate(const rocs_dca_cache_args* a, AttnPlan* pl) {
  if (!a) return ROCS_ERR_INVALID_ARG;
  int rc = cache_validate(a->cache);
  if (rc) return rc;
  if (a->R < 0 || a->q <= 0 || a->H <= 0 || a->max_pages < 0) return ROCS_ERR_INVALID_ARG;
  if (a->H % a->cache.heads) return ROCS_ERR_INVALID_ARG;
  if (!std::isfinite(a->scale) || a->scale < 0.0f) return ROCS_ERR_INVALID_ARG;
  if (a->R >= (int64_t(1) << 28) || a->q >= (int64_t(1) << 20) || a->H >= (int64_t(1) << 16) ||
      a->max_pages * a->cache.page >= (int64_t(1) << 30))
    return ROCS_ERR_UNSUPPORTED;
  if ((rc = check_csr_ext(a->cand_off_host, a->R, &pl->C))) return rc;
  if (pl->C * a->q * a->H >= (int64_t(1) << 31)) return ROCS_ERR_UNSUPPORTED;
  if (pl->C > 0) {
    if (!a->cand_off_dev || !a->seq_len || !a->q_ptr || !a->o_ptr || (a->max_pages > 0 && !a->page_table))
      return ROCS_ERR_INVALID_ARG;
    if (!al(a->q_ptr, 16) || !al(a->o_ptr, 16) || !al(a->lse_ptr, 4) || !al(a->cand_off_dev, 4) || !al(a->seq_len, 4) ||
        !al(a->page_table, 4) || !al(a->key_limit, 4))
      return ROCS_ERR_INVALID_ARG;
    const int64_t row = a->H * a->cache.dh;
    if (a->q_ld != 0 && a->q_ld < row) return ROCS_ERR_INVALID_ARG;
    if (a->q_ld % 8 || a->q_ld >= (int64_t(1) << 31)) return ROCS_ERR_UNSUPPORTED;
    // outputs that overlap the queries, the cache or each other: all are read after other parts' outputs are written
    const int64_t n = pl->C * a->q;
    const Span q = span(a->q_ptr, n, row, a->q_ld ? a->q_ld : row, 2), o = span(a->o_ptr, n, row, row, 2);
    const Span l = a->lse_ptr ? span(a->lse_ptr, n, a->H, a->H, 4) : Span{0, 0};
    Span c[4];
    cache_spans(a->cache, c);
    if (!apart(q, o) || !apart(q, l) || !apart(o, l)) return ROCS_ERR_INVALID_ARG;
    for (const Span& b : c)
      if (!apart(o, b) || !apart(l, b)) return ROCS_ERR_INVALID_ARG;
    const int64_t G = a->H / a->cache.heads;
    const bool wide = a->cache.dh == 128;
    const int64_t limit = wide ? kFewLimit128 : kFewLimit64, many = wide ? kManyCost128 : kManyCost64;
    const int64_t chunk = G > kMaxShared ? 1 : 2 * (128 / G) * G;
    int64_t all_few = 0, all_many = 0, mixed = 0, most = 0;
    for (int64_t r = 0; r < a->R; ++r) {
      const int64_t rows = (a->cand_off_host[r + 1] - a->cand_off_host[r]) * a->q * G;
      const int64_t f = kFewCost * ((rows + kFewRows - 1) / kFewRows), m = many * ((rows + chunk - 1) / chunk);
      all_few += f;
      all_many += m;
      mixed += rows <= limit ? f : m;
      if (rows > most) most = rows;
    }
    if (G > kMaxShared || (all_few <= all_many && 4 * all_few <= 5 * mixed)) pl->rows_hi = 0x7fffffff;
    else pl->rows_hi = 4 * all_many <= 5 * mixed ? 0 : (int)limit;
    // the rows that the first kernel sees at most (its unit size goes by them), and whether the second has work
    for (int64_t r = 0; r < a->R; ++r) {
      const int64_t rows = (a->cand_off_host[r + 1] - a->cand_off_host[r]) * a->q * G;
      if (rows <= pl->rows_hi && rows > pl->rows_few) pl->rows_few = (int)rows;
    }
    pl->grid_many = most > pl->rows_hi ? 1 : 0;
    const int sms = sm_count_ext();
    pl->grid_many *= sms;
    pl->grid_few = pl->rows_few ? cache_few_grid(sms) : 0;
  }
  const size_t part_few = 2 * (size_t)pl->grid_few * cache_few_part_bytes((int)a->cache.dh);
  const size_t part_many = 2 * (size_t)pl->grid_many * cache_many_part_bytes((int)a->cache.dh);
  pl->cnt_many = sizeof(WsHeader) + a256(sizeof(int) * (size_t)pl->grid_few);
  pl->zero = pl->cnt_many + a256(8 * sizeof(int) * (size_t)pl->grid_many);
  pl->bytes = pl->zero + (part_few > part_many ? part_few : part_many);  // one kernel after the other
  return ROCS_OK;
}

}  // namespace

extern "C" {

size_t rocs_dca_cache_workspace_size(const rocs_dca_cache_args* a) {
  AttnPlan pl;
  return attn_validate(a, &pl) == ROCS_OK ? pl.bytes : 0;
}

int rocs_dca_cache_forward(const rocs_dca_cache_args* a, rocs_stream_t stream) {
  AttnPlan pl;
  int rc = attn_validate(a, &pl);
  if (rc || (rc = workspace_validate(a->workspace, a->workspace_bytes, pl.bytes))) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(a->workspace);
  if (cudaMemsetAsync(ws, 0, pl.zero, st) != cudaSuccess) return ROCS_ERR_CUDA;
  CacheAttnParams p;
  std::memset(&p, 0, sizeof(p));
  p.c = cache_of(a->cache);
  p.q = static_cast<const __nv_bfloat16*>(a->q_ptr);
  p.o = static_cast<__nv_bfloat16*>(a->o_ptr);
  p.lse = a->lse_ptr;
  p.cand_off = a->cand_off_dev;
  p.seq_len = a->seq_len;
  p.table = a->page_table;
  p.key_limit = a->key_limit;
  p.q_ld = a->q_ld ? a->q_ld : a->H * a->cache.dh;
  p.R = (int)a->R;
  p.C = (int)pl.C;
  p.q_tokens = (int)a->q;
  p.H = (int)a->H;
  p.G = (int)(a->H / a->cache.heads);
  p.max_pages = (int)a->max_pages;
  p.capacity = a->cache.pages > 0 ? (int)(a->max_pages * a->cache.page) : 0;
  p.scale_log2 = a->scale * 1.4426950408889634f;
  p.ws = reinterpret_cast<WsHeader*>(ws);
  p.part = reinterpret_cast<float*>(ws + pl.zero);
  int launches = 0;
  if (pl.grid_few) {
    p.rows_lo = 0;
    p.rows_hi = pl.rows_hi;
    p.cnt = reinterpret_cast<int*>(ws + sizeof(WsHeader));
    if (launch_cache_few(p, (int)a->cache.dh, pl.rows_few, pl.grid_few, st) != cudaSuccess) return ROCS_ERR_CUDA;
    ++launches;
  }
  if (pl.grid_many) {
    CacheManyParams m;
    std::memset(&m, 0, sizeof(m));
    if (!tmap_bf16_3d_ext(&m.tm_q, p.q, (uint64_t)a->cache.dh, (uint64_t)a->H, (uint64_t)(pl.C * a->q), (uint64_t)a->cache.dh * 2,
                          (uint64_t)p.q_ld * 2, 64, (uint32_t)p.G, (uint32_t)(128 / p.G)))
      return ROCS_ERR_CUDA;
    m.a = p;
    m.a.rows_lo = pl.rows_hi;
    m.a.rows_hi = 0x7fffffff;
    m.a.cnt = reinterpret_cast<int*>(ws + pl.cnt_many);
    m.min_share = 2;
    m.wait_limit_ns = kDefaultWaitLimitNs;
    if (launch_cache_many(m, (int)a->cache.dh, pl.grid_many, st) != cudaSuccess) return ROCS_ERR_CUDA;
    ++launches;
  }
  set_last_launches(launches);
  return ROCS_OK;
}

size_t rocs_qk_norm_rope_workspace_size(const rocs_norm_rope_args* a) {
  return norm_rope_validate(a) == ROCS_OK ? sizeof(WsHeader) : 0;
}

int rocs_qk_norm_rope_forward(const rocs_norm_rope_args* a, rocs_stream_t stream) {
  int rc = norm_rope_validate(a);
  if (rc || (rc = workspace_validate(a->workspace, a->workspace_bytes, sizeof(WsHeader)))) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  NormRopeParams p;
  std::memset(&p, 0, sizeof(p));
  const int64_t rows[2] = {a->q.n * a->q.heads, a->k.n * a->k.heads};
  const int unroll = unroll_for(rows[0] + rows[1], a->dh, sm_count_ext(), kNormSets), per = unroll * rows_per_warp(a->dh);
  const rocs_norm_rope_side* s[2] = {&a->q, &a->k};
  for (int i = 0; i < 2; ++i) {
    const int64_t row = s[i]->heads * a->dh;
    p.side[i].x = s[i]->x;
    p.side[i].out = s[i]->out;
    p.side[i].pos = s[i]->pos;
    p.side[i].gamma = s[i]->gamma;
    p.side[i].beta = s[i]->beta;
    p.side[i].ld_x = s[i]->ld_x ? s[i]->ld_x : row;
    p.side[i].ld_out = s[i]->ld_out ? s[i]->ld_out : row;
    p.side[i].n = (int)s[i]->n;
    p.side[i].heads = (int)s[i]->heads;
    p.warps += (rows[i] + per - 1) / per;
    if (i == 0) p.warps0 = p.warps;
  }
  p.rope = a->rope;
  p.max_pos = (int)a->max_pos;
  p.rot = (int)a->rot;
  p.interleaved = a->interleaved != 0;
  p.norm = a->norm;
  p.eps = a->eps;
  p.ws = static_cast<WsHeader*>(a->workspace);
  if (cudaMemsetAsync(p.ws, 0, sizeof(WsHeader), st) != cudaSuccess) return ROCS_ERR_CUDA;
  if (p.warps > 0 && launch_norm_rope(p, (int)a->dh, a->dtype == ROCS_F32, unroll, st) != cudaSuccess) return ROCS_ERR_CUDA;
  set_last_launches(p.warps > 0 ? 1 : 0);
  return ROCS_OK;
}

int rocs_rope_table(float* table, int64_t max_pos, int64_t rot, double base, rocs_stream_t stream) {
  if (max_pos < 0 || rot <= 0 || !(base > 1.0) || !std::isfinite(base)) return ROCS_ERR_INVALID_ARG;
  if (rot % 16 || rot > 128 || max_pos >= (int64_t(1) << 31)) return ROCS_ERR_UNSUPPORTED;
  if (max_pos == 0) {
    set_last_launches(0);
    return ROCS_OK;
  }
  if (!table || !al(table, 16)) return ROCS_ERR_INVALID_ARG;
  if (launch_rope_table(table, max_pos, (int)rot, base, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
    return ROCS_ERR_CUDA;
  set_last_launches(1);
  return ROCS_OK;
}

size_t rocs_cache_workspace_size(const rocs_cache_move_args* a) {
  int64_t T;
  return move_validate(a, true, &T) == ROCS_OK ? sizeof(WsHeader) : 0;
}
int rocs_cache_append(const rocs_cache_move_args* a, rocs_stream_t stream) {
  return cache_move(a, true, reinterpret_cast<cudaStream_t>(stream));
}
int rocs_cache_read(const rocs_cache_move_args* a, rocs_stream_t stream) {
  return cache_move(a, false, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
