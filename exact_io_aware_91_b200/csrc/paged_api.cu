// Host side of the paged key/value cache in include/fa.h: argument checks and launches.
// No allocation and no synchronisation happen here.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "paged.h"

using namespace fa;

namespace {

constexpr int kMaxPages = 1 << 20;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// log2 of a supported page size, or -1.
int page_shift(int page_size) {
  for (int s = 3; s <= 10; ++s)
    if (page_size == (1 << s)) return s;
  return -1;
}

// Sizes and strides that fa_paged_attn and fa_pages_write share.  queries: H and scale count too.
fa_status check_paged(const fa_paged_problem* p, bool queries, bool* empty) {
  if (p == nullptr) return FA_ERR_INVALID_ARG;
  if (p->B < 0 || p->H_kv < 1 || p->T < 0 || p->num_pages < 0 || p->max_pages < 0 || p->table_stride < p->max_pages)
    return FA_ERR_INVALID_ARG;
  if (p->dtype != FA_BF16 && p->dtype != FA_F16) return FA_ERR_INVALID_ARG;
  if (queries) {
    if (p->H < 1 || p->H % p->H_kv != 0 || p->prefix_len < 0) return FA_ERR_INVALID_ARG;
    if (p->causal != 0 && p->causal != 1) return FA_ERR_INVALID_ARG;
    if (!(std::isfinite(p->scale) && p->scale > 0.f)) return FA_ERR_INVALID_ARG;
  }
  if (p->d != 64 && p->d != 128 && p->d != 256) return FA_ERR_UNSUPPORTED;
  if (page_shift(p->page_size) < 0 || p->num_pages > kMaxPages) return FA_ERR_UNSUPPORTED;
  for (const long long* st : {p->k_stride, p->v_stride})
    for (int i = 0; i < 3; ++i)
      if (st[i] < p->d || st[i] % 8 != 0 || st[i] >= (1ll << 38)) return FA_ERR_INVALID_ARG;
  const long long heads = queries ? p->H : p->H_kv;
  if ((long long)p->B * p->H_kv > (1 << 24) || heads > (1 << 16) || p->T > (1 << 24) ||
      (long long)p->B * heads > (1 << 24) || (long long)p->B * heads * p->T > 0x7fffffffLL / 2)
    return FA_ERR_UNSUPPORTED;
  if ((long long)p->max_pages * p->page_size > (1 << 30) || (queries && p->prefix_len > (1 << 30)) ||
      (long long)p->B * p->table_stride > (1ll << 40))
    return FA_ERR_UNSUPPORTED;
  *empty = p->B == 0 || p->T == 0;
  if (queries && !*empty) {
    // all (item, key tile) units, with one more per item, are counted in 32 bits
    const PagedWs w = paged_ws_layout(p->B, p->H, p->H_kv, p->T, p->d);
    const long long own = ((long long)p->max_pages * p->page_size + 63) / 64, pre = (p->prefix_len + 63ll) / 64;
    const long long groups = std::max(w.n_groups[0], w.n_groups[1]);
    if (w.own_items > 0x7fffffffLL / (own + pre + 1) || groups * p->H_kv > 0x7fffffffLL / (pre + 1))
      return FA_ERR_UNSUPPORTED;
  }
  return FA_OK;
}

fa_status to_status(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

// The table of the page operations; `t` is filled in apart from the error word.
fa_status check_table(const fa_page_table* pt, TableArgs* t) {
  if (pt == nullptr) return FA_ERR_INVALID_ARG;
  if (pt->rows < 0 || pt->max_pages < 0 || pt->num_pages < 0 || pt->table_stride < pt->max_pages)
    return FA_ERR_INVALID_ARG;
  const int shift = page_shift(pt->page_size);
  if (shift < 0 || pt->num_pages > kMaxPages || pt->rows > (1 << 24) ||
      (long long)pt->max_pages * pt->page_size > (1 << 30))
    return FA_ERR_UNSUPPORTED;
  t->table = pt->block_table;
  t->lens = pt->seq_lens;
  t->refs = pt->ref_counts;
  t->rows = pt->rows;
  t->max_pages = pt->max_pages;
  t->stride = pt->table_stride;
  t->page_shift = shift;
  t->num_pages = pt->num_pages;
  return FA_OK;
}
// Pointers of a table that is going to be used (rows, pages and entries may each be 0 of).
fa_status check_table_ptrs(const TableArgs& t) {
  if ((t.rows > 0 && (!t.lens || (t.max_pages > 0 && !t.table))) || (t.num_pages > 0 && !t.refs))
    return FA_ERR_INVALID_ARG;
  if (!aligned(t.table, 4) || !aligned(t.lens, 4) || !aligned(t.refs, 4)) return FA_ERR_MISALIGNED;
  return FA_OK;
}

fa_status check_planes(const fa_page_planes* pl) {
  if (pl == nullptr || pl->n_planes < 0 || pl->num_pages < 0 || pl->page_bytes < 0 ||
      pl->page_stride < pl->page_bytes || (pl->n_planes > 0 && pl->planes == nullptr))
    return FA_ERR_INVALID_ARG;
  if (pl->n_planes > kMaxPlanes || pl->num_pages > kMaxPages || pl->page_bytes > (1ll << 30) ||
      pl->page_stride > (1ll << 40))
    return FA_ERR_UNSUPPORTED;
  if (pl->page_bytes % 16 != 0 || pl->page_stride % 16 != 0) return FA_ERR_MISALIGNED;
  for (int i = 0; i < pl->n_planes; ++i) {
    if (pl->num_pages > 0 && pl->page_bytes > 0 && pl->planes[i] == nullptr) return FA_ERR_INVALID_ARG;
    if (!aligned(pl->planes[i], 16)) return FA_ERR_MISALIGNED;
  }
  return FA_OK;
}

// Calls fn(pointers, count, first) for every kPlanesPerLaunch planes; at least once if `tables`.
template <class F>
fa_status for_planes(const fa_page_planes* pl, bool tables, F fn) {
  const int n = pl->page_bytes > 0 && pl->num_pages > 0 ? pl->n_planes : 0;
  for (int at = 0; at < n || (at == 0 && tables); at += kPlanesPerLaunch) {
    PlanePtrs ptrs{};
    const int m = std::min(kPlanesPerLaunch, n - at);
    for (int i = 0; i < m; ++i) ptrs.p[i] = static_cast<uint8_t*>(pl->planes[at + i]);
    const cudaError_t e = fn(ptrs, m, at == 0);
    if (e != cudaSuccess) return FA_ERR_CUDA;
  }
  return FA_OK;
}

fa_status check_ws(const void* ws, size_t bytes, size_t need) {
  if (ws == nullptr || bytes < need) return FA_ERR_INVALID_ARG;
  return aligned(ws, 256) ? FA_OK : FA_ERR_MISALIGNED;
}

// fa_paged_attn; with give_up = n > 0 every CTA that has n segments gives up its waits from the n-th on.
fa_status paged_attn(const fa_paged_problem* pr, const void* q, const void* k_pages, const void* v_pages,
                     const int* block_table, const int* seq_lens, const int* prefix_table, void* o, float* lse,
                     void* workspace, size_t workspace_bytes, fa_stream_t stream, int give_up) {
  bool empty = false;
  fa_status st = check_paged(pr, true, &empty);
  if (st != FA_OK || empty) return st;
  if (!q || !o || !seq_lens || (pr->num_pages > 0 && (!k_pages || !v_pages)) ||
      (pr->max_pages > 0 && !block_table) || (pr->prefix_len > 0 && !prefix_table))
    return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(lse, 4) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(prefix_table, 4))
    return FA_ERR_MISALIGNED;
  if ((st = check_ws(workspace, workspace_bytes, fa_paged_attn_workspace_size(pr))) != FA_OK) return st;
  PagedParams p{};
  int num_sms = 0;
  if ((st = device_ready(&num_sms, &p.err)) != FA_OK) return st;
  const PagedWs w = paged_ws_layout(pr->B, pr->H, pr->H_kv, pr->T, pr->d);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int d = pr->d;
  p.table = block_table;
  p.lens = seq_lens;
  p.prefix_table = prefix_table;
  p.o = o;
  p.lse = lse;
  p.B = pr->B;
  p.H = pr->H;
  p.H_kv = pr->H_kv;
  p.T = pr->T;
  p.R = pr->H / pr->H_kv * pr->T;
  p.page_shift = page_shift(pr->page_size);
  p.num_pages = pr->num_pages;
  p.max_pages = pr->max_pages;
  p.table_stride = pr->table_stride;
  p.prefix_len = pr->prefix_len;
  p.causal = pr->causal;
  p.box_rows = std::min(pr->page_size, 32);
  p.packed = w.packed;
  p.n_rc = w.n_rc;
  p.own_few = w.own_few;
  // keys per tile: 128; 64 in the dense form at d = 256 (tensor memory), 256 in the few-rows form at d = 64
  const int few_kt = d == 64 ? 8 : 7, dense_kt = d == 256 ? 6 : 7;
  p.pre_few = prefix_few(w, p.H_kv, p.prefix_len, few_kt);
  p.seqs = w.packed ? w.seqs[p.pre_few] : 1;
  p.group_seqs = w.group_seqs[p.pre_few];
  p.n_groups = w.n_groups[p.pre_few];
  p.pre_rows = w.pre_rows[p.pre_few];
  p.own_kt = w.own_few ? few_kt : dense_kt;
  p.pre_kt = p.pre_few ? few_kt : dense_kt;
  p.pre_tiles = (pr->prefix_len + (1 << p.pre_kt) - 1) >> p.pre_kt;
  p.ctas = std::min(num_sms, kPagedMaxCtas);
  p.give_up = give_up;
  p.scale_log2 = pr->scale * 1.4426950408889634f;
  p.seg = reinterpret_cast<int2*>(ws + w.off_seg);
  p.own_ml = reinterpret_cast<float2*>(ws + w.off_own_ml);
  p.own_o = reinterpret_cast<float*>(ws + w.off_own_o);
  p.pre_ml = reinterpret_cast<float2*>(ws + w.off_pre_ml);
  p.pre_o = reinterpret_cast<float*>(ws + w.off_pre_o);

  typedef unsigned long long u64;
  const bool bf = pr->dtype == FA_BF16;
  PagedMaps maps;
  // q as (d, R rows, H_kv, B): a box takes the same rows of one sequence (own items) or of
  // p.seqs consecutive sequences (prefix items)
  const u64 row = 2ull * d, qd[4] = {(u64)d, (u64)p.R, (u64)p.H_kv, (u64)p.B};
  const u64 qs[3] = {row, row * p.R, row * p.R * p.H_kv};
  const unsigned box_q = (unsigned)std::min(p.R, 128);
  const unsigned own_box[4] = {64, box_q, 1, 1}, pre_box[4] = {64, box_q, 1, (unsigned)p.seqs};
  const unsigned kv_box[4] = {64, (unsigned)p.box_rows, 1, 1};
  // pages: (d, page_size, H_kv, num_pages); the page id after the last one reads zeros
  const u64 kd[4] = {(u64)d, (u64)pr->page_size, (u64)p.H_kv, (u64)std::max(p.num_pages, 1)};
  u64 ks[3], vs[3];
  for (int i = 0; i < 3; ++i) {
    ks[i] = 2ull * pr->k_stride[2 - i];
    vs[i] = 2ull * pr->v_stride[2 - i];
  }
  const void* kb = p.num_pages > 0 ? k_pages : q;
  const void* vb = p.num_pages > 0 ? v_pages : q;
  if (!make_tmap_4d(&maps.q_own, q, bf, qd, qs, own_box) || !make_tmap_4d(&maps.q_pre, q, bf, qd, qs, pre_box) ||
      !make_tmap_4d(&maps.k, kb, bf, kd, ks, kv_box) || !make_tmap_4d(&maps.v, vb, bf, kd, vs, kv_box))
    return FA_ERR_CUDA;
  return to_status(launch_paged_attn(maps, p, d, pr->dtype, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

size_t fa_paged_attn_workspace_size(const fa_paged_problem* pr) {
  bool empty = false;
  if (check_paged(pr, true, &empty) != FA_OK || empty) return 0;
  return paged_ws_layout(pr->B, pr->H, pr->H_kv, pr->T, pr->d).total;
}

fa_status fa_paged_attn(const fa_paged_problem* pr, const void* q, const void* k_pages, const void* v_pages,
                        const int* block_table, const int* seq_lens, const int* prefix_table, void* o, float* lse,
                        void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  return paged_attn(pr, q, k_pages, v_pages, block_table, seq_lens, prefix_table, o, lse, workspace, workspace_bytes,
                    stream, 0);
}

fa_status fa_selftest_paged_give_up(const fa_paged_problem* pr, const void* q, const void* k_pages,
                                    const void* v_pages, const int* block_table, const int* seq_lens,
                                    const int* prefix_table, void* o, float* lse, void* workspace,
                                    size_t workspace_bytes, int segment, fa_stream_t stream) {
  if (segment < 1) return FA_ERR_INVALID_ARG;
  return paged_attn(pr, q, k_pages, v_pages, block_table, seq_lens, prefix_table, o, lse, workspace, workspace_bytes,
                    stream, segment);
}

fa_status fa_pages_write(const fa_paged_problem* pr, const void* k, const void* v, void* k_pages, void* v_pages,
                         const int* block_table, const int* seq_lens, fa_stream_t stream) {
  bool empty = false;
  fa_status st = check_paged(pr, false, &empty);
  if (st != FA_OK || empty) return st;
  if (!k || !v || !seq_lens || (pr->num_pages > 0 && (!k_pages || !v_pages)) || (pr->max_pages > 0 && !block_table))
    return FA_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4))
    return FA_ERR_MISALIGNED;
  WriteArgs a{};
  int num_sms = 0;
  if ((st = device_ready(&num_sms, &a.err)) != FA_OK) return st;
  a.k = static_cast<const uint4*>(k);
  a.v = static_cast<const uint4*>(v);
  a.kp = static_cast<uint8_t*>(k_pages);
  a.vp = static_cast<uint8_t*>(v_pages);
  for (int i = 0; i < 3; ++i) {
    a.ks[i] = 2 * pr->k_stride[i];
    a.vs[i] = 2 * pr->v_stride[i];
  }
  a.table = block_table;
  a.lens = seq_lens;
  a.B = pr->B;
  a.H_kv = pr->H_kv;
  a.T = pr->T;
  a.d8 = pr->d / 8;
  a.table_stride = pr->table_stride;
  a.max_pages = pr->max_pages;
  a.page_shift = page_shift(pr->page_size);
  a.num_pages = pr->num_pages;
  return to_status(launch_pages_write(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t fa_pages_workspace_size(int rows, int num_pages) {
  if (rows < 0 || num_pages < 0) return 0;
  return pages_ws_layout(rows, num_pages).total;
}

fa_status fa_pages_copy(const fa_page_planes* planes, const int* src, const int* dst, int n, fa_stream_t stream) {
  fa_status st = check_planes(planes);
  if (st != FA_OK) return st;
  if (n < 0) return FA_ERR_INVALID_ARG;
  if (n == 0) return FA_OK;
  if (n > (1 << 24)) return FA_ERR_UNSUPPORTED;
  if (!src || !dst) return FA_ERR_INVALID_ARG;
  if (!aligned(src, 4) || !aligned(dst, 4)) return FA_ERR_MISALIGNED;
  int num_sms = 0, *err = nullptr;
  if ((st = device_ready(&num_sms, &err)) != FA_OK) return st;
  return for_planes(planes, true, [&](const PlanePtrs& ptrs, int m, bool) {
    return launch_pages_copy(ptrs, m, planes->page_bytes, planes->page_stride, src, dst, n, planes->num_pages,
                             num_sms, err, reinterpret_cast<cudaStream_t>(stream));
  });
}

fa_status fa_pages_reserve(const fa_page_table* table, const int* new_lens, void* workspace, size_t workspace_bytes,
                           fa_stream_t stream) {
  TableArgs t{};
  fa_status st = check_table(table, &t);
  if (st != FA_OK) return st;
  if (t.rows == 0) return FA_OK;
  if (!new_lens) return FA_ERR_INVALID_ARG;
  if ((st = check_table_ptrs(t)) != FA_OK) return st;
  if (!aligned(new_lens, 4)) return FA_ERR_MISALIGNED;
  if ((st = check_ws(workspace, workspace_bytes, fa_pages_workspace_size(t.rows, t.num_pages))) != FA_OK) return st;
  int num_sms = 0;
  if ((st = device_ready(&num_sms, &t.err)) != FA_OK) return st;
  return to_status(launch_pages_reserve(t, new_lens, static_cast<uint8_t*>(workspace),
                                        reinterpret_cast<cudaStream_t>(stream)));
}

fa_status fa_pages_fork(const fa_page_planes* planes, const fa_page_table* table, const int* parents,
                        const int* children, int n, void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  TableArgs t{};
  fa_status st = check_table(table, &t);
  if (st != FA_OK) return st;
  if ((st = check_planes(planes)) != FA_OK) return st;
  if (planes->num_pages != t.num_pages || n < 0 || n > t.rows) return FA_ERR_INVALID_ARG;
  if (n == 0) return FA_OK;
  if (!parents || !children) return FA_ERR_INVALID_ARG;
  if ((st = check_table_ptrs(t)) != FA_OK) return st;
  if (!aligned(parents, 4) || !aligned(children, 4)) return FA_ERR_MISALIGNED;
  if ((st = check_ws(workspace, workspace_bytes, fa_pages_workspace_size(t.rows, t.num_pages))) != FA_OK) return st;
  int num_sms = 0;
  if ((st = device_ready(&num_sms, &t.err)) != FA_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (launch_pages_fork_plan(t, parents, children, n, ws, s) != cudaSuccess) return FA_ERR_CUDA;
  return for_planes(planes, true, [&](const PlanePtrs& ptrs, int m, bool first) {
    return launch_pages_fork_apply(t, ptrs, m, planes->page_bytes, planes->page_stride, parents, children, n, first,
                                   num_sms, ws, s);
  });
}

fa_status fa_pages_free(const fa_page_table* table, const int* rows, int n, fa_stream_t stream) {
  TableArgs t{};
  fa_status st = check_table(table, &t);
  if (st != FA_OK) return st;
  if (n < 0) return FA_ERR_INVALID_ARG;
  if (n == 0 || t.rows == 0) return FA_OK;
  if (!rows) return FA_ERR_INVALID_ARG;
  if ((st = check_table_ptrs(t)) != FA_OK) return st;
  if (!aligned(rows, 4)) return FA_ERR_MISALIGNED;
  int num_sms = 0;
  if ((st = device_ready(&num_sms, &t.err)) != FA_OK) return st;
  return to_status(launch_pages_free(t, rows, n, reinterpret_cast<cudaStream_t>(stream)));
}

fa_status fa_pages_compact(const fa_page_planes* planes, const fa_page_table* table, int* block_table_out,
                           int* ref_counts_out, int* page_map, void* workspace, size_t workspace_bytes,
                           fa_stream_t stream) {
  TableArgs t{};
  fa_status st = check_table(table, &t);
  if (st != FA_OK) return st;
  if ((st = check_planes(planes)) != FA_OK) return st;
  if (planes->num_pages != t.num_pages) return FA_ERR_INVALID_ARG;
  if ((t.num_pages > 0 && (!ref_counts_out || !page_map)) || (t.rows > 0 && t.max_pages > 0 && !block_table_out))
    return FA_ERR_INVALID_ARG;
  if ((st = check_table_ptrs(t)) != FA_OK) return st;
  if (!aligned(block_table_out, 4) || !aligned(ref_counts_out, 4) || !aligned(page_map, 4)) return FA_ERR_MISALIGNED;
  if ((st = check_ws(workspace, workspace_bytes, fa_pages_workspace_size(t.rows, t.num_pages))) != FA_OK) return st;
  int num_sms = 0;
  if ((st = device_ready(&num_sms, &t.err)) != FA_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (launch_pages_compact_plan(t, ref_counts_out, page_map, ws, s) != cudaSuccess) return FA_ERR_CUDA;
  return for_planes(planes, true, [&](const PlanePtrs& ptrs, int m, bool first) {
    return launch_pages_compact_apply(t, ptrs, m, planes->page_bytes, planes->page_stride, block_table_out, page_map,
                                      first, num_sms, ws, s);
  });
}

}  // extern "C"
