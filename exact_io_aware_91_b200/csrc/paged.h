// Internal interface of the paged key/value cache: the launches behind the fa_paged_attn and
// fa_pages_* entry points (checks of arguments in paged_api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "../../include/fa.h"

namespace fa {

// What the kernels of the paged cache record in the error word besides the codes of sm100.cuh: an index out
// of its range, too few free pages.  (Kept apart from the headers of the dense kernels: recorded counters
// of those are void once their shared headers change.)
enum : int { kDevIndex = FA_ERR_INDEX, kDevNoPages = FA_ERR_NO_PAGES };

// Checks the current device; its multiprocessor count and the address of its error word.
fa_status device_ready(int* num_sms, int** err);

// ------------------------------------------------------------------ page operations
constexpr int kMaxPlanes = 1024;
constexpr int kPlanesPerLaunch = 256;  // plane pointers travel as a kernel parameter (2 KB)

struct PlanePtrs {
  uint8_t* p[kPlanesPerLaunch];
};

struct TableArgs {
  int* table;
  int* lens;
  int* refs;
  int rows, max_pages, stride, page_shift, num_pages;
  int* err;
};

struct PagesWs {  // layout of the page operations' workspace
  size_t off_rows, off_pages, total;
};
inline PagesWs pages_ws_layout(int rows, int num_pages) {
  auto align256 = [](size_t x) { return (x + 255) & ~(size_t)255; };
  PagesWs w{};
  w.off_rows = 256;                                        // control block first
  w.off_pages = w.off_rows + align256((size_t)rows * 16);  // int[4][rows]
  w.total = w.off_pages + align256((size_t)num_pages * 8); // int[2][num_pages]
  return w;
}

struct WriteArgs {
  const uint4* k;
  const uint4* v;
  uint8_t* kp;
  uint8_t* vp;
  long long ks[3], vs[3];  // bytes between pages, heads, tokens
  const int* table;
  const int* lens;
  int B, H_kv, T, d8, table_stride, max_pages, page_shift, num_pages;
  int* err;
};

cudaError_t launch_pages_write(const WriteArgs& a, cudaStream_t s);
cudaError_t launch_pages_copy(const PlanePtrs& pl, int n_planes, long long page_bytes, long long page_stride,
                              const int* src, const int* dst, int n, int num_pages, int num_sms, int* err,
                              cudaStream_t s);
cudaError_t launch_pages_free(const TableArgs& t, const int* rows, int n, cudaStream_t s);
cudaError_t launch_pages_reserve(const TableArgs& t, const int* new_lens, uint8_t* ws, cudaStream_t s);
cudaError_t launch_pages_fork_plan(const TableArgs& t, const int* parents, const int* children, int n, uint8_t* ws,
                                   cudaStream_t s);
// one launch per kPlanesPerLaunch planes; the first one (with_tables) also writes tables and counts
cudaError_t launch_pages_fork_apply(const TableArgs& t, const PlanePtrs& pl, int n_planes, long long page_bytes,
                                    long long page_stride, const int* parents, const int* children, int n,
                                    bool with_tables, int num_sms, uint8_t* ws, cudaStream_t s);
cudaError_t launch_pages_compact_plan(const TableArgs& t, int* refs_out, int* page_map, uint8_t* ws, cudaStream_t s);
cudaError_t launch_pages_compact_apply(const TableArgs& t, const PlanePtrs& pl, int n_planes, long long page_bytes,
                                       long long page_stride, int* table_out, const int* page_map, bool with_tables,
                                       int num_sms, uint8_t* ws, cudaStream_t s);

// ------------------------------------------------------------------ attention over pages
constexpr int kPagedMaxCtas = 148;  // persistent CTAs of the attention kernel (one per multiprocessor)
constexpr int kFewRows = 32;        // items of at most this many rows take the products with swapped operands
constexpr int kItemCost = 1;        // an item's own cost in the division of the line, in key tiles

struct PagedParams {
  const int* table;
  const int* lens;
  const int* prefix_table;
  void* o;
  float* lse;
  int B, H, H_kv, T, R;  // R = H / H_kv * T query rows share a key/value head: they lie side by side in q and o
  int page_shift, num_pages, max_pages, table_stride, prefix_len;
  int causal;
  int box_rows;    // tokens per TMA box of K and V
  int packed;      // 1: the prefix has work items of its own, each for the rows of several sequences
  int own_few, pre_few;  // own / prefix items have at most kFewRows rows
  int seqs;        // packed: sequences per query tile of a prefix item
  int group_seqs;  // packed: sequences per prefix item
  int pre_rows;    // packed: rows of a prefix item's slot
  int n_rc;        // row chunks of a (sequence, key/value head)
  int n_groups;    // packed: prefix items per key/value head
  int own_kt, pre_kt;  // log2 of the keys per tile
  int pre_tiles;   // key tiles of the prefix
  int ctas;        // grid
  int give_up;     // self-test: n > 0 raises a CTA's abort flag at its n-th segment
  float scale_log2;
  // partial results (unnormalised O, and the maximum and sum of each row), see PagedWs
  int2* seg;       // own items: first and last part of the line that holds the item
  float2* own_ml;
  float* own_o;
  float2* pre_ml;
  float* pre_o;
  int* err;
};

// Workspace of fa_paged_attn.  Own items are numbered (b * n_rc + rc) * H_kv + h, prefix items
// h * n_groups + group.  An item that one CTA works on alone has the slot of its number (own items:
// only when a prefix part has to be joined, otherwise the result is written at once); the part c of
// the line that starts an item and does not end it has slot n_items + 2 c + 1, one that goes on with
// an item begun in another part slot n_items + 2 c.
struct PagedWs {
  int item_rows;  // rows of an item: 256 (two 128-row tiles), d = 256: 128
  int slot_rows;  // rows of an own slot
  int packed, own_few, n_rc;
  // prefix items in the dense form [0] and in the few-rows form [1]: sequences per query tile and per
  // item, items per key/value head, rows of a slot
  int seqs[2], group_seqs[2], n_groups[2], pre_rows[2];
  long long own_items, own_slots, pre_slots[2];
  size_t off_seg, off_own_ml, off_own_o, off_pre_ml, off_pre_o, total;
};
inline PagedWs paged_ws_layout(int B, int H, int H_kv, int T, int d) {
  auto align256 = [](size_t x) { return (x + 255) & ~(size_t)255; };
  PagedWs w{};
  const long long R = (long long)H / H_kv * T;
  w.item_rows = d == 256 ? 128 : 256;
  w.packed = R <= 128;
  w.own_few = R <= kFewRows;
  w.n_rc = (int)((R + w.item_rows - 1) / w.item_rows);
  w.slot_rows = (int)(R < w.item_rows ? R : w.item_rows);
  w.own_items = (long long)B * w.n_rc * H_kv;
  w.own_slots = (w.packed ? w.own_items : 0) + 2 * kPagedMaxCtas;
  size_t pre_slot_rows = 0;
  for (int f = 0; f < 2; ++f) {
    if (!(f ? w.own_few : w.packed)) continue;
    w.seqs[f] = (int)((f ? kFewRows : 128) / R);
    if (w.seqs[f] > B) w.seqs[f] = B;
    w.group_seqs[f] = f ? w.seqs[f] : w.seqs[f] * (w.item_rows / 128);
    w.n_groups[f] = (B + w.group_seqs[f] - 1) / w.group_seqs[f];
    w.pre_rows[f] = f ? kFewRows : w.item_rows;
    w.pre_slots[f] = (long long)w.n_groups[f] * H_kv + 2 * kPagedMaxCtas;
    const size_t rows = (size_t)w.pre_slots[f] * w.pre_rows[f];
    if (rows > pre_slot_rows) pre_slot_rows = rows;
  }
  w.off_seg = 0;
  w.off_own_ml = align256((size_t)w.own_items * sizeof(int2));
  w.off_own_o = w.off_own_ml + align256((size_t)w.own_slots * w.slot_rows * sizeof(float2));
  w.off_pre_ml = w.off_own_o + align256((size_t)w.own_slots * w.slot_rows * d * sizeof(float));
  w.off_pre_o = w.off_pre_ml + align256(pre_slot_rows * sizeof(float2));
  w.total = w.off_pre_o + align256(pre_slot_rows * d * sizeof(float));
  return w;
}

// Whether an own item's note of its parts (PagedParams::seg) names parts of the line at all.  A CTA that
// gave up a wait leaves the notes of its items unwritten: they are what the workspace held before, and the
// joining kernel must not go where they point.
__host__ __device__ inline bool parts_known(int first, int last, int ctas) {
  return 0 <= first && first <= last && last < ctas;
}

// The form of the prefix items: the few-rows form reads the prefix once for every 32 rows, the dense
// form once for every 256, but next to own items in the few-rows form it is a phase of its own (its
// code and its first tiles, some 10 us of each CTA).  Up to 4 few-rows units per CTA are cheaper:
// 24 sequences of 5 rows and 16 heads (d = 64) over 2000 tokens, 3.5 units each, take 63 us against 65
// in the dense form, over 4000 tokens 68 against 67.  (Measured there only; other head dims and row
// counts have other tiles, and take the same limit.)
inline int prefix_few(const PagedWs& w, int H_kv, int prefix_len, int few_kt) {
  if (!w.packed || !w.own_few) return 0;
  const long long tiles = ((long long)prefix_len + (1 << few_kt) - 1) >> few_kt;
  return w.n_groups[1] == 1 || w.n_groups[1] * H_kv * tiles <= 4 * kPagedMaxCtas;
}

struct PagedMaps {
  CUtensorMap q_own, q_pre, k, v;
};
// (64 columns x rows) boxes with the 128-byte swizzle over a 4-D 16-bit tensor; strides in bytes
bool make_tmap_4d(CUtensorMap* m, const void* base, bool bf16, const unsigned long long (&dims)[4],
                  const unsigned long long (&strides)[3], const unsigned (&box)[4]);
cudaError_t launch_paged_attn(const PagedMaps& maps, const PagedParams& p, int d, int dtype, cudaStream_t s);

}  // namespace fa
