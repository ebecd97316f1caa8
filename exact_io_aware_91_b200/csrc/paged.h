// Internal interface of the paged key/value cache: the launches behind the fa_paged_attn and
// fa_pages_* entry points (checks of arguments in paged_api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "../../include/fa.h"

namespace fa {

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
  w.off_pages = w.off_rows + align256((size_t)rows * 8);   // int[2][rows]
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
struct PagedParams {
  const void* q;
  const void* k;
  const void* v;
  void* o;
  float* lse;
  const int* table;
  const int* lens;
  const int* prefix_table;
  long long ks[3], vs[3];  // elements between pages, heads, tokens
  int B, H, H_kv, T;
  int page_shift, num_pages, max_pages, table_stride, prefix_len;
  int causal;
  float scale_log2;
  int* err;
};
cudaError_t launch_paged_attn(const PagedParams& p, int d, int dtype, cudaStream_t s);

}  // namespace fa
