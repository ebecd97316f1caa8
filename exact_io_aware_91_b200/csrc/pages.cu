// Operations on the pages of a key/value cache: writing tokens, copying, reserving, forking,
// freeing and compacting pages.  All state lives in device arrays (block table, lengths,
// reference counts), so nothing here synchronises with the host.
//
// Data movement is bound by memory: every byte is read once and written once with 16-byte
// accesses, several in flight per thread.  Decisions (which pages are free, who gets which) are
// made by ONE block per call: the k-th page asked for is the k-th lowest free id, which is a
// running count over ref_counts, and a single block scans 4096 counts per step without any
// exchange between blocks.  Results are therefore the same on every run.  Counts change by
// integer atomics, whose order does not matter.
#include <algorithm>

#include "paged.h"
#include "sm100.cuh"

namespace fa {
namespace {

constexpr int kPlan = 1024;  // threads of the deciding block
constexpr int kPer = 4;      // consecutive counts per thread and step

__device__ __forceinline__ void report(int* err, int code) { atomicExch(err, code); }

// Exclusive running sum over the block's threads; *total is the block's sum.
__device__ __forceinline__ int block_scan(int v, int* total, int* smem) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) smem[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = smem[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w += y;
    }
    smem[lane] = w;
  }
  __syncthreads();
  const int base = warp > 0 ? smem[warp - 1] : 0;
  *total = smem[31];
  __syncthreads();  // smem may be used again
  return base + x - v;
}

// Entries that a row of length `len` owns (at most max_pages).
__device__ __forceinline__ int owned_entries(int len, const TableArgs& t) {
  if (len <= 0) return 0;
  const int n = (int)(((long long)len + (1 << t.page_shift) - 1) >> t.page_shift);
  return n < t.max_pages ? n : t.max_pages;
}

// The ids of the `want` lowest free pages (or of all, if there are fewer) into ids[]; returns how many.
__device__ __forceinline__ int find_free(const TableArgs& t, int want, int* ids, int* smem) {
  int found = 0;
  for (int base = 0; base < t.num_pages && found < want; base += kPlan * kPer) {
    const int p0 = base + threadIdx.x * kPer;
    bool is_free[kPer];
    int n = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      is_free[i] = p0 + i < t.num_pages && t.refs[p0 + i] == 0;
      n += is_free[i] ? 1 : 0;
    }
    int total;
    int rank = found + block_scan(n, &total, smem);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (is_free[i]) {
        if (rank < want) ids[rank] = p0 + i;
        ++rank;
      }
    found += total;
  }
  return found < want ? found : want;
}

// ---------------------------------------------------------------------------- data movement
// `bytes` (a multiple of 16) from src to dst by the whole block, four 16-byte loads in flight per thread.
__device__ __forceinline__ void block_copy(uint8_t* dst, const uint8_t* src, long long bytes) {
  const uint4* s = reinterpret_cast<const uint4*>(src);
  uint4* d = reinterpret_cast<uint4*>(dst);
  const long long n = bytes >> 4;
  long long i = threadIdx.x;
  for (; i + 3 * blockDim.x < n; i += 4 * blockDim.x) {
    uint4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) x[u] = s[i + u * blockDim.x];
#pragma unroll
    for (int u = 0; u < 4; ++u) d[i + u * blockDim.x] = x[u];
  }
  for (; i < n; i += blockDim.x) d[i] = s[i];
}

struct Chunks {  // a page's bytes in every plane, cut into pieces for one block each
  long long page_bytes, page_stride;
  int n_planes, per_page;  // pieces per page and plane
  long long piece;         // bytes of a piece (the last of a page may be smaller)
};
__device__ __forceinline__ void copy_piece(const PlanePtrs& pl, const Chunks& c, int piece, int src, int dst) {
  const int plane = piece / c.per_page, part = piece - plane * c.per_page;
  const long long at = part * c.piece;
  const long long bytes = c.page_bytes - at < c.piece ? c.page_bytes - at : c.piece;
  uint8_t* base = pl.p[plane] + at;
  block_copy(base + dst * c.page_stride, base + src * c.page_stride, bytes);
}

// ---------------------------------------------------------------------------- write
__global__ void __launch_bounds__(256) fa_pages_write_kernel(const WriteArgs a) {
  const long long n = (long long)a.B * a.H_kv * a.T * a.d8;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const uint4 xk = a.k[i], xv = a.v[i];
  const int c = (int)(i % a.d8);
  long long r = i / a.d8;
  const int tok = (int)(r % a.T);
  r /= a.T;
  const int h = (int)(r % a.H_kv), b = (int)(r / a.H_kv);
  const int len = a.lens[b];
  const long long pos = (long long)len - a.T + tok;
  if (len < 0 || pos < 0) return;
  const long long e = pos >> a.page_shift;
  if (e >= a.max_pages) {
    report(a.err, kDevIndex);
    return;
  }
  const int page = a.table[(long long)b * a.table_stride + e];
  if (page < 0 || page >= a.num_pages) {
    report(a.err, kDevIndex);
    return;
  }
  const long long in = pos & ((1 << a.page_shift) - 1);
  *reinterpret_cast<uint4*>(a.kp + page * a.ks[0] + h * a.ks[1] + in * a.ks[2] + c * 16) = xk;
  *reinterpret_cast<uint4*>(a.vp + page * a.vs[0] + h * a.vs[1] + in * a.vs[2] + c * 16) = xv;
}

// ---------------------------------------------------------------------------- copy
// blockIdx.x: pair; blockIdx.y: share of the pair's pieces.  Every block first looks through the
// whole list for pairs that exclude its own.
__global__ void __launch_bounds__(256) fa_pages_copy_kernel(const __grid_constant__ PlanePtrs pl, const Chunks c,
                                                            const int* __restrict__ src,
                                                            const int* __restrict__ dst, int n, int num_pages,
                                                            int* err) {
  const int me = blockIdx.x;
  const int s = src[me], d = dst[me];
  if (s < 0 || d < 0 || s == d) return;
  if (s >= num_pages || d >= num_pages) {
    if (threadIdx.x == 0) report(err, kDevIndex);
    return;
  }
  int bad = 0;
  for (int j = threadIdx.x; j < n; j += 256) {
    const int sj = src[j], dj = dst[j];
    if (sj < 0 || dj < 0 || sj == dj || sj >= num_pages || dj >= num_pages) continue;
    if ((j < me && dj == d) || sj == d) bad = 1;
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) report(err, kDevIndex);
    return;
  }
  for (int piece = blockIdx.y; piece < c.n_planes * c.per_page; piece += gridDim.y) copy_piece(pl, c, piece, s, d);
}

// The same for lists of kLongList pairs and more: a block takes `per` (at most kCopyList) consecutive pairs
// and looks through the list once for all of them, with a hash table of their destinations; a block per
// pair reads n^2 entries.  Measured (this form / a block per pair, us): pages of 4 KB in one plane 52 / 69
// at 8192 pairs, 214 / 710 at 32768, 407 / 2677 at 65536; of 16 KB in four planes 411 / 355 at 16384,
// 609 / 577 at 24576, 834 / 866 at 32768, 1665 / 2923 at 65536.
constexpr int kLongList = 1 << 15;
constexpr int kCopyList = 1024, kCopyTable = 2048;  // at most half full

__global__ void __launch_bounds__(256) fa_pages_copy_list_kernel(const __grid_constant__ PlanePtrs pl, const Chunks c,
                                                                 const int* __restrict__ src,
                                                                 const int* __restrict__ dst, int n, int per,
                                                                 int num_pages, int* err) {
  __shared__ int s_src[kCopyList], s_dst[kCopyList];
  // first[h]: the first of the block's pairs whose destination is key[h], -1 once a pair of the list excludes it
  __shared__ int key[kCopyTable], first[kCopyTable];
  const int start = blockIdx.x * per, m = min(per, n - start);
  for (int h = threadIdx.x; h < kCopyTable; h += 256) key[h] = -1, first[h] = n;
  __syncthreads();
  auto hash = [](int id) -> int { return (int)(((unsigned)id * 2654435761u) >> 21); };
  auto find = [&](int id) -> int {
    int h = hash(id);
    while (key[h] != id) {
      if (key[h] < 0) return -1;
      h = (h + 1) & (kCopyTable - 1);
    }
    return h;
  };
  for (int i = threadIdx.x; i < m; i += 256) {
    const int s = src[start + i];
    int d = dst[start + i];
    if (s < 0 || s == d) d = -1;
    if (d >= 0 && (s >= num_pages || d >= num_pages)) {
      report(err, kDevIndex);
      d = -1;
    }
    s_src[i] = s;
    s_dst[i] = d;
    if (d < 0) continue;
    int h = hash(d);
    for (int k; (k = atomicCAS(&key[h], -1, d)) != -1 && k != d;) h = (h + 1) & (kCopyTable - 1);
    atomicMin(&first[h], i);
  }
  __syncthreads();
  for (int j = threadIdx.x; j < n; j += 256) {
    const int sj = src[j], dj = dst[j];
    if (sj < 0 || dj < 0 || sj == dj || sj >= num_pages || dj >= num_pages) continue;
    int h = find(sj);
    if (h >= 0) atomicExch(&first[h], -1);
    if (j < start && (h = find(dj)) >= 0) atomicExch(&first[h], -1);
  }
  __syncthreads();
  for (int i = 0; i < m; ++i) {
    const int d = s_dst[i];
    if (d < 0) continue;
    if (first[find(d)] < i) {
      if (threadIdx.x == 0) report(err, kDevIndex);
      continue;
    }
    for (int piece = 0; piece < c.n_planes * c.per_page; ++piece) copy_piece(pl, c, piece, s_src[i], d);
  }
}

// ---------------------------------------------------------------------------- free
__global__ void __launch_bounds__(kPlan) fa_pages_free_kernel(const TableArgs t, const int* __restrict__ rows) {
  __shared__ int s_len;
  const int row = rows[blockIdx.x];
  if (row < 0) return;
  if (row >= t.rows) {
    if (threadIdx.x == 0) report(t.err, kDevIndex);
    return;
  }
  // the exchange gives the length to one block: a second mention of the row finds -1
  if (threadIdx.x == 0) s_len = atomicExch(&t.lens[row], -1);
  __syncthreads();
  const int len = s_len;
  const int n = owned_entries(len, t);
  if (threadIdx.x == 0 && (long long)len > ((long long)t.max_pages << t.page_shift)) report(t.err, kDevIndex);
  int* mine = t.table + (long long)row * t.stride;
  for (int e = threadIdx.x; e < n; e += kPlan) {
    const int page = mine[e];
    mine[e] = -1;
    if (page < 0 || page >= t.num_pages) {
      report(t.err, kDevIndex);
    } else if (atomicSub(&t.refs[page], 1) <= 0) {
      atomicAdd(&t.refs[page], 1);  // nobody counted this entry: the count stays 0
      report(t.err, kDevIndex);
    }
  }
}

// ---------------------------------------------------------------------------- reserve
// Workspace: rows[0][b] = pages asked for by the rows before b; pages[] = the free pages found.
__global__ void __launch_bounds__(kPlan) fa_pages_reserve_kernel(const TableArgs t, const int* __restrict__ new_lens,
                                                                 int* before, int* ids) {
  __shared__ int smem[32];
  auto asked = [&](int b, int& have, int& len) -> int {
    const int cur = t.lens[b];
    len = new_lens[b];
    have = owned_entries(cur, t);
    if (len <= (cur > 0 ? cur : 0)) return 0;
    if ((long long)len > ((long long)t.max_pages << t.page_shift)) {
      len = -1;  // does not fit the table
      return 0;
    }
    return owned_entries(len, t) - have;
  };
  int want = 0;
  for (int base = 0; base < t.rows; base += kPlan) {
    const int b = base + threadIdx.x;
    int have = 0, len = 0, total;
    const int need = b < t.rows ? asked(b, have, len) : 0;
    // beyond num_pages nothing can be granted: the running sum saturates there (num_pages <= 2^20,
    // so 1024 rows' sum stays below 2^31)
    const int cap = t.num_pages + 1;
    const int ex = want + block_scan(min(need, cap), &total, smem);
    if (b < t.rows) before[b] = min(ex, cap);
    want = min(want + total, cap);
  }
  __syncthreads();
  const int found = want > 0 ? find_free(t, want < t.num_pages ? want : t.num_pages, ids, smem) : 0;
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int b = warp; b < t.rows; b += kPlan / 32) {
    int have, len;
    const int need = asked(b, have, len);
    const int first = before[b];
    __syncwarp();  // every lane has read the row's length before lane 0 changes it
    if (len < 0) {
      if (lane == 0 && new_lens[b] >= 0) report(t.err, kDevIndex);
      continue;
    }
    if (need > 0 && (long long)first + need > found) {
      if (lane == 0) report(t.err, kDevNoPages);
      continue;
    }
    int* mine = t.table + (long long)b * t.stride;
    for (int i = lane; i < need; i += 32) {
      const int page = ids[first + i];
      mine[have + i] = page;
      t.refs[page] = 1;
    }
    if (lane == 0 && len > (t.lens[b] > 0 ? t.lens[b] : 0)) t.lens[b] = len;
  }
}

// ---------------------------------------------------------------------------- fork
// Workspace rows[0][i]: what the plan decided for fork i: the id of its fresh last page, kNoTail
// when all the parent's pages are full, kLeftOut when it does not happen.  rows[1]: running need.
// rows[2][r]: the first fork whose child is row r, rows[3][r]: whether r is the parent of one; set for the
// rows of the list only, so that a fork is held against all others in a constant number of steps (against
// the list itself, 2^18 forks would take 2^36 compares of this one block).
constexpr int kNoTail = -1, kLeftOut = -2;

__global__ void __launch_bounds__(kPlan) fa_pages_fork_plan_kernel(const TableArgs t, const int* __restrict__ parents,
                                                                   const int* __restrict__ children, int n, int* fresh,
                                                                   int* before, int* first, int* is_parent, int* ids) {
  __shared__ int smem[32];
  for (int i = threadIdx.x; i < n; i += kPlan) {
    const int par = parents[i], chi = children[i];
    if (par < 0 || chi < 0) continue;
    if (par < t.rows) first[par] = n, is_parent[par] = 0;
    if (chi < t.rows) first[chi] = n, is_parent[chi] = 0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlan) {
    const int par = parents[i], chi = children[i];
    if (par < 0 || chi < 0) continue;
    if (par < t.rows) is_parent[par] = 1;
    if (chi < t.rows) atomicMin(&first[chi], i);
  }
  __syncthreads();
  int want = 0;
  for (int base = 0; base < n; base += kPlan) {
    const int i = base + threadIdx.x;
    int par = -1, chi = -1;
    if (i < n) {
      par = parents[i];
      chi = children[i];
    }
    bool takes = i < n && par >= 0 && chi >= 0;
    if (takes) {
      bool bad = par >= t.rows || chi >= t.rows || par == chi;
      if (!bad) {
        const int len = t.lens[par];
        bad = len < 0 || (long long)len > ((long long)t.max_pages << t.page_shift) || t.lens[chi] > 0;
        // a parent that is also a child, a child that is also a parent, a child forked before
        bad = bad || first[par] < n || is_parent[chi] != 0 || first[chi] < i;
      }
      if (bad) report(t.err, kDevIndex);
      takes = !bad;
    }
    const int need = takes && (t.lens[par] & ((1 << t.page_shift) - 1)) != 0 ? 1 : 0;
    int total;
    const int ex = want + block_scan(need, &total, smem);
    if (i < n) {
      before[i] = ex;
      fresh[i] = !takes ? kLeftOut : need ? 0 : kNoTail;
    }
    want += total;
  }
  __syncthreads();
  const int found = want > 0 ? find_free(t, want < t.num_pages ? want : t.num_pages, ids, smem) : 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlan)
    if (fresh[i] == 0) {
      if (before[i] < found) {
        fresh[i] = ids[before[i]];
        t.refs[fresh[i]] = 1;
      } else {
        fresh[i] = kLeftOut;
        report(t.err, kDevNoPages);
      }
    }
}

// blockIdx.x: fork; blockIdx.y = 0 (with_tables): its row of the table and the counts; the other
// blocks: shares of its last page's pieces.
__global__ void __launch_bounds__(256) fa_pages_fork_apply_kernel(const TableArgs t, const __grid_constant__ PlanePtrs pl,
                                                                  const Chunks c, const int* __restrict__ parents,
                                                                  const int* __restrict__ children, int with_tables,
                                                                  const int* __restrict__ fresh) {
  const int i = blockIdx.x;
  const int tail = fresh[i];
  if (tail == kLeftOut) return;
  const int par = parents[i], chi = children[i];
  const int len = t.lens[par];
  const int full = len >> t.page_shift;
  const int* from = t.table + (long long)par * t.stride;
  if (with_tables && blockIdx.y == 0) {
    int* to = t.table + (long long)chi * t.stride;
    for (int e = threadIdx.x; e < full; e += 256) {
      const int page = from[e];
      to[e] = page;
      if (page < 0 || page >= t.num_pages)
        report(t.err, kDevIndex);
      else
        atomicAdd(&t.refs[page], 1);
    }
    if (threadIdx.x == 0) {
      if (tail >= 0) to[full] = tail;
      t.lens[chi] = len;
    }
    return;
  }
  if (tail < 0) return;
  const int src = from[full];
  if (src < 0 || src >= t.num_pages) {
    if (threadIdx.x == 0) report(t.err, kDevIndex);
    return;
  }
  for (int piece = blockIdx.y - with_tables; piece < c.n_planes * c.per_page; piece += gridDim.y - with_tables)
    copy_piece(pl, c, piece, src, tail);
}

// ---------------------------------------------------------------------------- compact
// Workspace: ctrl[0] = number of moves; pages[]: holes (num_pages / 2), movers (num_pages / 2),
// movers' counts (num_pages / 2).  There are as many free ids below n_live as live ids from it on,
// at most num_pages / 2 of each.
__global__ void __launch_bounds__(kPlan) fa_pages_compact_plan_kernel(const TableArgs t, int* refs_out, int* map,
                                                                      int* ctrl, int* holes, int* movers,
                                                                      int* counts) {
  __shared__ int smem[32];
  int live = 0;
  for (int p = threadIdx.x; p < t.num_pages; p += kPlan) live += t.refs[p] > 0 ? 1 : 0;
  int n_live;
  block_scan(live, &n_live, smem);
  int n_holes = 0, n_movers = 0;
  for (int base = 0; base < t.num_pages; base += kPlan * kPer) {
    const int p0 = base + threadIdx.x * kPer;
    int ref[kPer];
    int both = 0;  // holes in the low half, movers in the high half (at most 4096 each)
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int p = p0 + i;
      ref[i] = p < t.num_pages ? t.refs[p] : 0;
      if (p < n_live && ref[i] <= 0) both += 1;
      if (p >= n_live && ref[i] > 0) both += 1 << 16;
    }
    int total;
    const int ex = block_scan(both, &total, smem);
    int h = n_holes + (ex & 0xffff), m = n_movers + (ex >> 16);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int p = p0 + i;
      if (p >= t.num_pages) break;
      if (p < n_live) {
        map[p] = ref[i] > 0 ? p : -1;
        refs_out[p] = ref[i] > 0 ? ref[i] : 0;
        if (ref[i] <= 0) holes[h++] = p;
      } else {
        map[p] = -1;
        refs_out[p] = 0;
        if (ref[i] > 0) {
          movers[m] = p;
          counts[m++] = ref[i];
        }
      }
    }
    n_holes += total & 0xffff;
    n_movers += total >> 16;
  }
  __syncthreads();
  for (int k = threadIdx.x; k < n_movers; k += kPlan) {
    map[movers[k]] = holes[k];
    refs_out[holes[k]] = counts[k];
  }
  if (threadIdx.x == 0) ctrl[0] = n_movers;
}

__global__ void __launch_bounds__(256) fa_pages_compact_apply_kernel(const TableArgs t, const __grid_constant__ PlanePtrs pl,
                                                                     const Chunks c, int* table_out,
                                                                     const int* __restrict__ map, int with_tables,
                                                                     const int* __restrict__ ctrl,
                                                                     const int* __restrict__ holes,
                                                                     const int* __restrict__ movers) {
  if (with_tables)
    for (int b = blockIdx.x; b < t.rows; b += gridDim.x) {
      const int n = owned_entries(t.lens[b], t);
      const int* from = t.table + (long long)b * t.stride;
      int* to = table_out + (long long)b * t.stride;
      for (int e = threadIdx.x; e < t.max_pages; e += 256) {
        int page = from[e];
        if (e < n) {
          if (page >= 0 && page < t.num_pages)
            page = map[page];
          else
            report(t.err, kDevIndex);
        }
        to[e] = page;
      }
    }
  const int per_move = c.n_planes * c.per_page;
  const long long n = (long long)ctrl[0] * per_move;
  for (long long i = blockIdx.x; i < n; i += gridDim.x) {
    const int k = (int)(i / per_move);
    copy_piece(pl, c, (int)(i - (long long)k * per_move), movers[k], holes[k]);
  }
}

// Pieces of `target` bytes or less, one at least (a page may have no bytes, or a call no planes).
Chunks cut(int n_planes, long long page_bytes, long long page_stride, long long target) {
  Chunks c{};
  c.page_bytes = page_bytes;
  c.page_stride = page_stride;
  c.n_planes = n_planes;
  c.per_page = (int)((page_bytes + target - 1) / target);
  if (c.per_page < 1) c.per_page = 1;
  c.piece = ((page_bytes + c.per_page - 1) / c.per_page + 15) & ~15ll;
  return c;
}
constexpr long long kPiece = 16384;  // one piece: four 16-byte loads of each of 256 threads

}  // namespace

cudaError_t launch_pages_write(const WriteArgs& a, cudaStream_t s) {
  const long long n = (long long)a.B * a.H_kv * a.T * a.d8;
  fa_pages_write_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_pages_copy(const PlanePtrs& pl, int n_planes, long long page_bytes, long long page_stride,
                              const int* src, const int* dst, int n, int num_pages, int num_sms, int* err,
                              cudaStream_t s) {
  const Chunks c = cut(n_planes, page_bytes, page_stride, kPiece);
  // blocks enough to fill the device eight deep, not more: each of them reads the whole list
  if (n >= kLongList) {
    const int per = std::min((n + 8 * num_sms - 1) / (8 * num_sms), kCopyList);
    fa_pages_copy_list_kernel<<<(n + per - 1) / per, 256, 0, s>>>(pl, c, src, dst, n, per, num_pages, err);
    return cudaGetLastError();
  }
  const long long pieces = (long long)n_planes * c.per_page;
  long long y = (8ll * num_sms + n - 1) / n;
  y = y > pieces ? pieces : y;
  y = y < 1 ? 1 : y;  // without pieces the list is checked all the same
  fa_pages_copy_kernel<<<dim3(n, (unsigned)(y < 65535 ? y : 65535)), 256, 0, s>>>(pl, c, src, dst, n, num_pages, err);
  return cudaGetLastError();
}

cudaError_t launch_pages_free(const TableArgs& t, const int* rows, int n, cudaStream_t s) {
  fa_pages_free_kernel<<<n, kPlan, 0, s>>>(t, rows);
  return cudaGetLastError();
}

cudaError_t launch_pages_reserve(const TableArgs& t, const int* new_lens, uint8_t* ws, cudaStream_t s) {
  const PagesWs w = pages_ws_layout(t.rows, t.num_pages);
  fa_pages_reserve_kernel<<<1, kPlan, 0, s>>>(t, new_lens, reinterpret_cast<int*>(ws + w.off_rows),
                                              reinterpret_cast<int*>(ws + w.off_pages));
  return cudaGetLastError();
}

cudaError_t launch_pages_fork_plan(const TableArgs& t, const int* parents, const int* children, int n, uint8_t* ws,
                                   cudaStream_t s) {
  const PagesWs w = pages_ws_layout(t.rows, t.num_pages);
  int* rows = reinterpret_cast<int*>(ws + w.off_rows);
  const size_t r = (size_t)t.rows;
  fa_pages_fork_plan_kernel<<<1, kPlan, 0, s>>>(t, parents, children, n, rows, rows + r, rows + 2 * r, rows + 3 * r,
                                                reinterpret_cast<int*>(ws + w.off_pages));
  return cudaGetLastError();
}

cudaError_t launch_pages_fork_apply(const TableArgs& t, const PlanePtrs& pl, int n_planes, long long page_bytes,
                                    long long page_stride, const int* parents, const int* children, int n,
                                    bool with_tables, int num_sms, uint8_t* ws, cudaStream_t s) {
  const PagesWs w = pages_ws_layout(t.rows, t.num_pages);
  const Chunks c = cut(n_planes, page_bytes, page_stride, kPiece);
  const long long pieces = (long long)n_planes * c.per_page;
  long long y = (8ll * num_sms + n - 1) / n;
  y = (y < 1 ? 1 : y > pieces ? pieces : y) + (with_tables ? 1 : 0);
  fa_pages_fork_apply_kernel<<<dim3(n, (unsigned)(y < 65535 ? y : 65535)), 256, 0, s>>>(
      t, pl, c, parents, children, with_tables ? 1 : 0, reinterpret_cast<const int*>(ws + w.off_rows));
  return cudaGetLastError();
}

cudaError_t launch_pages_compact_plan(const TableArgs& t, int* refs_out, int* page_map, uint8_t* ws, cudaStream_t s) {
  const PagesWs w = pages_ws_layout(t.rows, t.num_pages);
  int* lists = reinterpret_cast<int*>(ws + w.off_pages);
  const int half = t.num_pages / 2;
  fa_pages_compact_plan_kernel<<<1, kPlan, 0, s>>>(t, refs_out, page_map, reinterpret_cast<int*>(ws), lists,
                                                   lists + half, lists + 2 * half);
  return cudaGetLastError();
}

cudaError_t launch_pages_compact_apply(const TableArgs& t, const PlanePtrs& pl, int n_planes, long long page_bytes,
                                       long long page_stride, int* table_out, const int* page_map, bool with_tables,
                                       int num_sms, uint8_t* ws, cudaStream_t s) {
  const PagesWs w = pages_ws_layout(t.rows, t.num_pages);
  const Chunks c = cut(n_planes, page_bytes, page_stride, kPiece);
  const int* lists = reinterpret_cast<const int*>(ws + w.off_pages);
  fa_pages_compact_apply_kernel<<<8 * num_sms, 256, 0, s>>>(t, pl, c, table_out, page_map, with_tables ? 1 : 0,
                                                            reinterpret_cast<const int*>(ws), lists,
                                                            lists + t.num_pages / 2);
  return cudaGetLastError();
}

}  // namespace fa
