// Attention of the newest tokens of every sequence over a paged key/value cache, with a prefix
// that the whole batch shares:
//   o = softmax(scale q [K_prefix; K_own]^T) [V_prefix; V_own]
//
// The softmax splits over any parts of the keys: part c gives a row's maximum m_c, sum l_c of
// 2^(s - m_c) and unnormalised O_c = sum 2^(s - m_c) v; with M = max m_c,
//   o = sum 2^(m_c - M) O_c / sum 2^(m_c - M) l_c.
//
// Work items.  The R = H / H_kv * T query rows of a sequence that share a key/value head lie side
// by side in q.  An OWN item is up to 256 of them (two 128-row tiles; d = 256: one tile, because two
// 256-column accumulators do not fit in tensor memory) against the sequence's own keys.  A PREFIX
// item packs the rows of as many sequences as two tiles hold against the shared keys, so each
// prefix key is read once for all of them and the products are dense.  With R > 128 the rows of
// one sequence fill tiles by themselves: then own items go over the prefix keys first and there are
// no prefix items.
//
// Split.  A unit is one item and one key tile (128 keys; d = 256: 64).  The units of all own items
// are one line, cut into equal parts for the persistent CTAs (one per multiprocessor), and so are
// those of the prefix items; a CTA walks its part of both lines.  So ragged lengths load all
// multiprocessors equally, without the host knowing them: every CTA adds up the lengths itself.  A part
// that covers an item only partly leaves (m, l, O) in the workspace, and a second kernel joins
// the parts of each row in the order of the line (the same on every run).  CTAs with an odd
// number walk the own line first: own items wait for memory (each key is used for R rows only),
// prefix items for the tensor core, and the two overlap across the device.
//
// In a CTA: warp 0 looks up pages and streams K and V tiles with TMA into a ring, one box per
// piece of a page (16 to 32 lanes issue one box each); warp 1 issues the tensor-core products, S of
// a step two steps ahead of its P V, across items; two warpgroups of softmax warps take the steps
// in turn, each with an S (then P) buffer and an O accumulator of its own in tensor memory.  With
// two query tiles a key tile is two steps, one per tile; with one tile the warpgroups take
// alternate key tiles and join their two partial results in the end.  A single query row costs a
// 128-row product: at 128 keys 0.5 us of tensor core against 1.5 us that a multiprocessor's share
// of the memory bandwidth takes for the keys, so the padding is not what bounds it.
//
// What lies behind a sequence's last token in a page never enters: its scores are masked, and the rows of
// the V tile are set to zero in shared memory (0 x NaN would be NaN).  P is rounded to the 16-bit
// type for the second product (it is at most 2^8, the running maximum may lag the true one by
// less than 8 in base 2); sums, maxima and O are fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged.h"
#include "sm100.cuh"

namespace fa {
namespace {

template <int D>
struct PLayout {
  static constexpr int KT = D == 256 ? 64 : 128;     // keys per tile
  static constexpr int NWG = D == 256 ? 1 : 2;       // softmax warpgroups = O accumulators = query tiles
  static constexpr int KCH = D / 64;                 // 128-byte column chunks per row
  static constexpr int QCHUNK = 128 * 128;           // one chunk of a query tile
  static constexpr int QTILE = KCH * QCHUNK;
  static constexpr int CHUNK = KT * 128;             // one chunk of a K or V tile
  static constexpr int SLOT = KCH * CHUNK;
  static constexpr int NS = D == 64 ? 12 : 5;        // ring slots
  static constexpr int THREADS = 128 + 128 * NWG;
  static constexpr int OFF_KV = NWG * QTILE;
  static constexpr int OFF_STAT = OFF_KV + NS * SLOT;  // float2[128]: a warpgroup's m and l for the other
  static constexpr int OFF_BAR = OFF_STAT + 1024;
  static constexpr int BAR_Q_FULL = 0;                 // [2]
  static constexpr int BAR_Q_EMPTY = 2;                // [2]
  static constexpr int BAR_S_FULL = 4;                 // [2]
  static constexpr int BAR_P_FULL = 6;                 // [2]
  static constexpr int BAR_O_FULL = 8;                 // [2]
  static constexpr int BAR_O_FREE = 10;                // [2]
  static constexpr int BAR_STAT_FULL = 12, BAR_STAT_EMPTY = 13, BAR_PV_DONE = 14, BAR_MMA_DONE = 15;
  static constexpr int BAR_KV_FULL = 16;               // [NS]
  static constexpr int BAR_KV_EMPTY = 16 + NS;         // [NS]
  static constexpr int NBAR = 16 + 2 * NS;
  static constexpr int OFF_START = OFF_BAR + NBAR * 8; // Start
  static constexpr int OFF_SCAN = OFF_START + 48;      // long long[12]
  static constexpr int OFF_TMEM_SLOT = OFF_SCAN + 96;
  static constexpr int OFF_ABORT = OFF_TMEM_SLOT + 8;
  static constexpr int SMEM_ALLOC = OFF_ABORT + 8 + 1024;
  static_assert(SMEM_ALLOC <= 232448, "shared memory per CTA");
  static_assert(NS >= 4, "S of a step is issued two steps ahead: two K and two V tiles are held at once");
  static __host__ __device__ constexpr uint32_t T_S(int i) { return i * KT; }
  static __host__ __device__ constexpr uint32_t T_O(int i) { return 256 + i * D; }
  static_assert(2 * KT <= 256 && 256 + NWG * D <= 512, "tensor memory columns");
};

// registers: the producer and product warps give theirs to the two softmax warpgroups
constexpr uint32_t kRegsLaunch = 168, kRegsLow = 72, kRegsHigh = 216;
static_assert(kRegsLow + 2 * kRegsHigh <= 3 * kRegsLaunch, "register split exceeds the launch budget");

__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > kWaitLimitNs) break;
  }
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* m, int c0, int c1, int c2, int c3,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}

__device__ __forceinline__ long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// ---------------------------------------------------------------------------- the two lines of units
// Own tokens of sequence b, at most what its row of the table holds; negative: no sequence.
__device__ __forceinline__ int own_len(const PagedParams& p, int b) {
  const int len = p.lens[b];
  const long long room = (long long)p.max_pages << p.page_shift;
  return len <= room ? len : (int)room;
}

// Own keys that some row of chunk rc sees (rows run over heads, then tokens).
template <int ITEM>
__device__ __forceinline__ int own_visible(const PagedParams& p, int len, int rc) {
  if (len <= 0 || !p.causal || p.n_rc == 1) return len < 0 ? 0 : len;
  const int r0 = rc * ITEM, n = min(ITEM, p.R - r0);
  const int t0 = r0 % p.T;
  const int last = t0 + n >= p.T ? p.T - 1 : t0 + n - 1;
  return max(0, len - p.T + last + 1);
}

// Key tiles of an own item: the prefix's first where it has no items of its own.
template <int KT>
__device__ __forceinline__ int own_tiles(const PagedParams& p, int len, int visible) {
  if (len < 0) return 0;
  return (p.packed ? 0 : p.pre_tiles) + (visible + KT - 1) / KT;
}

template <int D>
__device__ long long units_of(const PagedParams& p, int b) {
  using L = PLayout<D>;
  const int len = own_len(p, b);
  long long n = 0;
  for (int rc = 0; rc < p.n_rc; ++rc) n += own_tiles<L::KT>(p, len, own_visible<128 * L::NWG>(p, len, rc));
  return n * p.H_kv;
}

// A line of n units is cut into line_parts(n) parts, none of them empty: part c has the units from
// part_begin(c) on, and unit u is in part part_of(u).  The own line's parts go to the CTAs in falling
// order, so that a short prefix line and a short own line fall to different CTAs.
__device__ __forceinline__ int line_parts(const PagedParams& p, long long n) {
  return n < p.ctas ? (int)n : p.ctas;
}
__device__ __forceinline__ long long part_begin(long long n, int parts, int c) { return n * c / parts; }
__device__ __forceinline__ int part_of(long long n, int parts, long long u) {
  return (int)(((u + 1) * parts - 1) / n);
}

struct Start {  // where a CTA's part of the own line begins
  long long total;  // units of the whole line
  long long left;   // units of this CTA
  int b, rc, hk, tile;
};

// One item, or the part of it that falls into a CTA's part of the line.
struct Seg {
  bool own;
  int b, rc, hk;    // prefix: b is the first sequence of tile 0
  int len;          // own: the sequence's length
  int visible;      // own: keys seen by some row
  int t0, t1, nt;   // key tiles t0 .. t1 - 1 of nt
  bool pair;        // two query tiles
  int steps;
};

// Walks a CTA's segments; every role does so for itself.
template <int D>
struct Walk {
  using L = PLayout<D>;
  const PagedParams& p;
  long long pre_u, pre_end, own_left;
  int b, rc, hk, tile;
  int cur_b;
  int len;
  bool own_first;

  __device__ Walk(const PagedParams& p_, const Start& s) : p(p_) {
    const long long n = p.packed ? (long long)p.n_groups * p.H_kv * p.pre_tiles : 0;
    const int parts = line_parts(p, n), c = blockIdx.x;
    pre_u = c < parts ? part_begin(n, parts, c) : 0;
    pre_end = c < parts ? part_begin(n, parts, c + 1) : 0;
    own_left = s.left;
    b = s.b;
    rc = s.rc;
    hk = s.hk;
    tile = s.tile;
    cur_b = -1;
    len = 0;
    own_first = (blockIdx.x & 1) != 0;
  }
  __device__ bool next(Seg& s) {
    if (own_first && own_left > 0) return next_own(s);
    if (pre_u < pre_end) {
      const int item = (int)(pre_u / p.pre_tiles);
      s.own = false;
      s.hk = item / p.n_groups;
      s.b = (item - s.hk * p.n_groups) * p.seqs * L::NWG;
      s.rc = 0;
      s.len = s.visible = 0;
      s.nt = p.pre_tiles;
      s.t0 = (int)(pre_u - (long long)item * p.pre_tiles);
      s.t1 = (int)min((long long)s.nt, s.t0 + (pre_end - pre_u));
      s.pair = L::NWG == 2 && s.b + p.seqs < p.B;
      s.steps = (s.t1 - s.t0) * (s.pair ? 2 : 1);
      pre_u += s.t1 - s.t0;
      return true;
    }
    return own_left > 0 && next_own(s);
  }
  __device__ bool next_own(Seg& s) {
    for (; b < p.B;) {
      if (cur_b != b) {
        len = own_len(p, b);
        cur_b = b;
      }
      const int vis = own_visible<128 * L::NWG>(p, len, rc);
      const int nt = own_tiles<L::KT>(p, len, vis);
      if (nt > 0) {
        s.own = true;
        s.b = b;
        s.rc = rc;
        s.hk = hk;
        s.len = len;
        s.visible = vis;
        s.nt = nt;
        s.t0 = tile;
        s.t1 = (int)min((long long)nt, tile + own_left);
        s.pair = L::NWG == 2 && p.R - rc * 256 > 128;
        s.steps = (s.t1 - s.t0) * (s.pair ? 2 : 1);
        own_left -= s.t1 - s.t0;
        if (s.t1 < nt) {
          tile = s.t1;
          return true;
        }
      }
      tile = 0;
      // past this item; an item without tiles has none for the other heads either
      if (nt == 0 || ++hk == p.H_kv) {
        hk = 0;
        if (++rc == p.n_rc) {
          rc = 0;
          ++b;
        }
      }
      if (nt > 0) return true;
    }
    own_left = 0;  // the lengths changed under the call: stop instead of running past the batch
    return false;
  }
};

// Key tile `t` of a segment: whether it is the prefix's, its first token there and its tokens.
struct TileInfo {
  bool pre;
  int k0, n;
};
template <int KT>
__device__ __forceinline__ TileInfo tile_info(const PagedParams& p, const Seg& s, int t) {
  TileInfo x;
  const int lead = s.own ? (p.packed ? 0 : p.pre_tiles) : p.pre_tiles;
  x.pre = t < lead;
  x.k0 = (x.pre ? t : t - lead) * KT;
  x.n = min(KT, (x.pre ? p.prefix_len : s.visible) - x.k0);
  return x;
}

// ---------------------------------------------------------------------------- softmax step
template <bool BF>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  return BF ? pack_bf16(a, b) : pack_f16(a, b);
}

// One step of a row: S from tensor memory, keys from `lim` on masked, running maximum, O rescaled
// when the maximum has moved by 2^8 or more, P back over S.  `ready` waits until O may be touched.
template <int D, bool BF, class Ready>
__device__ __forceinline__ bool softmax_step(uint32_t tS, uint32_t tO, float sl2, int lim, bool first, float& m,
                                             float& l, Ready ready) {
  constexpr int KT = PLayout<D>::KT;
  float x[KT];
  {
    uint32_t u[KT / 32][32];
#pragma unroll
    for (int c = 0; c < KT / 32; ++c) tmem_ld32(tS + 32 * c, u[c]);
    tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < KT / 32; ++c)
#pragma unroll
      for (int i = 0; i < 32; ++i) x[32 * c + i] = __uint_as_float(u[c][i]);
  }
  if (__any_sync(0xffffffffu, lim < KT)) {
#pragma unroll
    for (int c = 0; c < KT; ++c)
      if (c >= lim) x[c] = -INFINITY;
  }
  float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
  for (int c = 4; c + 7 < KT; c += 8)
#pragma unroll
    for (int i = 0; i < 4; ++i) mx[i] = max3f(mx[i], x[c + 2 * i], x[c + 2 * i + 1]);
#pragma unroll
  for (int i = 0; i < 4; ++i) mx[i] = fmaxf(mx[i], x[KT - 4 + i]);
  const float m_new = fmaxf(m, fmaxf(max3f(mx[0], mx[1], mx[2]), mx[3]) * sl2);
  const float m_use = (m_new - m > 8.0f) ? m_new : m;
  const float alpha = (m_use == m) ? 1.0f : ex2_approx(m - m_use);  // 0 while nothing was visible before
  const float neg_m = m_use == -INFINITY ? 0.0f : -m_use;           // nothing visible yet: every P is 0
  if (!first && __any_sync(0xffffffffu, alpha != 1.0f)) {
    if (!ready()) return false;
    tc_fence_after();
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      uint32_t u[32];
      tmem_ld32(tO + 32 * c, u);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * alpha);
      tmem_st32(tO + 32 * c, u);
    }
  }
  uint64_t sa = 0, sb = 0;
#pragma unroll
  for (int h = 0; h < KT / 64; ++h) {
    uint32_t pk[32];
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      float* e = &x[64 * h + 2 * i];
      fma2(e[0], e[1], sl2, neg_m);
      fma2(e[2], e[3], sl2, neg_m);
#pragma unroll
      for (int k = 0; k < 4; ++k) e[k] = ex2_approx(e[k]);
      pk[i] = pack16<BF>(e[0], e[1]);
      pk[i + 1] = pack16<BF>(e[2], e[3]);
      asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sa) : "l"(f2pack(e[0], e[1])));
      asm("add.rn.f32x2 %0, %0, %1;" : "+l"(sb) : "l"(f2pack(e[2], e[3])));
    }
    tmem_st32(tS + 32 * h, pk);
  }
  float s0, s1, s2, s3;
  f2unpack(sa, s0, s1);
  f2unpack(sb, s2, s3);
  l = fmaf(l, alpha, (s0 + s1) + (s2 + s3));
  m = m_use;
  return true;
}

// ---------------------------------------------------------------------------- attention
template <int D, bool BF>
__global__ void __launch_bounds__(PLayout<D>::THREADS, 1)
    fa_paged_attn_sm100_kernel(const __grid_constant__ PagedMaps maps, const __grid_constant__ PagedParams p) {
  using L = PLayout<D>;
  constexpr int KT = L::KT, NWG = L::NWG, NS = L::NS, ITEM = 128 * NWG;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  auto bar = [&](int i) -> uint32_t { return base + L::OFF_BAR + 8u * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + L::OFF_ABORT);
  const WaitCtx wctx{abort_flag, p.err};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Start& start = *reinterpret_cast<Start*>(gbase + L::OFF_START);

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(L::BAR_Q_FULL + i), 1);
      mbar_init(bar(L::BAR_Q_EMPTY + i), 1);
      mbar_init(bar(L::BAR_S_FULL + i), 1);
      mbar_init(bar(L::BAR_P_FULL + i), 128);
      mbar_init(bar(L::BAR_O_FULL + i), 1);
      mbar_init(bar(L::BAR_O_FREE + i), 128);
    }
    mbar_init(bar(L::BAR_STAT_FULL), 128);
    mbar_init(bar(L::BAR_STAT_EMPTY), 128);
    mbar_init(bar(L::BAR_PV_DONE), 1);
    mbar_init(bar(L::BAR_MMA_DONE), 1);
    for (int i = 0; i < NS; ++i) {
      mbar_init(bar(L::BAR_KV_FULL + i), 1);
      mbar_init(bar(L::BAR_KV_EMPTY + i), 1);
    }
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(base + L::OFF_TMEM_SLOT, 512);
    tmem_relinquish();
  }
  // ---- this CTA's part of the own line: every thread adds up the units of its share of the
  // sequences, the block scans the sums, and the thread whose share holds the part's first unit finds it
  {
    long long* scan = reinterpret_cast<long long*>(gbase + L::OFF_SCAN);
    const int per = (int)ceil_div(p.B, L::THREADS);
    const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += units_of<D>(p, b);
    long long x = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) scan[warp] = x;
    if (threadIdx.x == 0) start.left = 0;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < L::THREADS / 32; ++w) {
      if (w < warp) before += scan[w];
      total += scan[w];
    }
    before += x - mine;
    const int parts = line_parts(p, total), part = p.ctas - 1 - (int)blockIdx.x;
    const long long lo = part < parts ? part_begin(total, parts, part) : 0;
    const long long hi = part < parts ? part_begin(total, parts, part + 1) : 0;
    if (hi > lo && before <= lo && lo < before + mine) {
      long long skip = lo - before;
      for (int b = b0; b < b1; ++b) {
        const long long n = units_of<D>(p, b);
        if (skip >= n) {
          skip -= n;
          continue;
        }
        const int len = own_len(p, b);
        for (int rc = 0; rc < p.n_rc; ++rc) {
          const int nt = own_tiles<KT>(p, len, own_visible<ITEM>(p, len, rc));
          if (skip >= (long long)nt * p.H_kv) {
            skip -= (long long)nt * p.H_kv;
            continue;
          }
          start.b = b;
          start.rc = rc;
          start.hk = (int)(skip / nt);
          start.tile = (int)(skip - (long long)start.hk * nt);
          start.left = hi - lo;
          break;
        }
        break;
      }
    }
    if (threadIdx.x == 0) start.total = total;
    if (blockIdx.x == 0)  // lengths that the table cannot hold
      for (int b = b0; b < b1; ++b)
        if (p.lens[b] > ((long long)p.max_pages << p.page_shift)) atomicExch(p.err, kDevIndex);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gbase + L::OFF_TMEM_SLOT);
  Walk<D> walk(p, start);
  Seg sg;

  if (warp == 0) {
    // ===================================================== page lookup and TMA
    if constexpr (NWG == 2) regs_dec<kRegsLow>();
    const int per_chunk = KT / p.box_rows;      // boxes per column chunk of a tile
    const int chunk = lane / per_chunk, piece = lane - chunk * per_chunk;
    const bool has_box = chunk < L::KCH;
    const int row0 = piece * p.box_rows;        // first token of this lane's box inside the tile
    const uint32_t box_bytes = (uint32_t)p.box_rows * 128u;
    const int page_mask = (1 << p.page_shift) - 1;
    const int no_page = max(p.num_pages, 1);    // reads zeros
    long long kv = 0, issued = 0;  // key tiles and ring slots filled so far
    int q_count[2] = {0, 0}, region = 0;
    bool ok = true;
    // the page of this lane's box in tile t
    auto look_up = [&](const Seg& s, int t) -> int {
      const TileInfo x = tile_info<KT>(p, s, t);
      if (!has_box || row0 >= x.n) return no_page;
      const int e = (x.k0 + row0) >> p.page_shift;
      const int page = x.pre ? p.prefix_table[e] : p.table[(long long)s.b * p.table_stride + e];
      if (page >= 0 && page < p.num_pages) return page;
      atomicExch(p.err, kDevIndex);
      return no_page;
    };
    while (ok && walk.next(sg)) {
      int page = look_up(sg, sg.t0);
      // Q: one region for a single tile (the other one keeps the previous item's), both for two tiles
      for (int w = 0; w < (sg.pair ? 2 : 1) && ok; ++w) {
        const int rg = sg.pair ? w : region;
        if (q_count[rg] > 0 && !(ok = mbar_wait(bar(L::BAR_Q_EMPTY + rg), (q_count[rg] - 1) & 1, wctx))) break;
        const int rows = min(p.R, 128) * (sg.own ? 1 : p.seqs);
        if (lane == 0) mbar_arrive_expect_tx(bar(L::BAR_Q_FULL + rg), (uint32_t)rows * 128u * L::KCH);
        __syncwarp();
        if (lane < L::KCH)
          tma_load_4d(base + rg * L::QTILE + lane * L::QCHUNK, sg.own ? &maps.q_own : &maps.q_pre, lane * 64,
                      sg.own ? sg.rc * ITEM + w * 128 : 0, sg.hk, sg.own ? sg.b : sg.b + w * p.seqs,
                      bar(L::BAR_Q_FULL + rg));
        ++q_count[rg];
      }
      if (NWG == 2 && !sg.pair) region ^= 1;
      for (int t = sg.t0; t < sg.t1 && ok; ++t, ++kv) {
        const TileInfo x = tile_info<KT>(p, sg, t);
        const int cur = page;
        if (t + 1 < sg.t1) page = look_up(sg, t + 1);
        const int boxes = (x.n + p.box_rows - 1) / p.box_rows;
        for (int v = 0; v < 2; ++v) {
          const long long i = 2 * kv + v;
          const int st = (int)(i % NS);
          if (!(ok = mbar_wait(bar(L::BAR_KV_EMPTY + st), ((uint32_t)(i / NS) & 1u) ^ 1u, wctx))) break;
          if (lane == 0) mbar_arrive_expect_tx(bar(L::BAR_KV_FULL + st), boxes * box_bytes * L::KCH);
          __syncwarp();
          if (has_box && row0 < x.n)
            tma_load_4d(base + L::OFF_KV + st * L::SLOT + chunk * L::CHUNK + row0 * 128, v ? &maps.v : &maps.k,
                        chunk * 64, (x.k0 + row0) & page_mask, sg.hk, cur, bar(L::BAR_KV_FULL + st));
          ++issued;
        }
        if (!ok) break;
      }
    }
    // every copy asked for has landed before the CTA may end (at once, unless a wait gave up)
    for (long long i = issued > NS ? issued - NS : 0; i < issued; ++i)
      drain_wait(bar(L::BAR_KV_FULL + (int)(i % NS)), (uint32_t)(i / NS) & 1u);
    for (int rg = 0; rg < 2; ++rg)
      if (q_count[rg] > 0) drain_wait(bar(L::BAR_Q_FULL + rg), (q_count[rg] - 1) & 1);
  } else if (warp == 1) {
    // ===================================================== products
    if constexpr (NWG == 2) regs_dec<kRegsLow>();
    const uint32_t leader = elect_one();
    constexpr uint32_t idesc_qk = make_idesc(128, KT, BF, false, false);
    constexpr uint32_t idesc_pv = make_idesc(128, D, BF, false, true);
    const uint64_t dQ0 = make_sdesc_sw128(base, 16, 1024);
    const uint64_t dK0 = make_sdesc_sw128(base + L::OFF_KV, 16, 1024);
    const uint64_t dV0 = make_sdesc_sw128(base + L::OFF_KV, L::CHUNK, 1024);
    bool ok = true;
    // S side: its own walk, two steps ahead of the P V side
    Seg a;
    a.steps = 0;
    int a_step = 0, a_region = 0, q_use[2] = {0, 0};
    long long a_kv = 0, a_total = 0;  // key tiles of earlier segments; steps so far
    bool a_more = true;
    auto issue_s = [&]() -> bool {
      if (!a_more) return true;
      if (a_step == a.steps) {
        a_kv += a.steps > 0 ? a.t1 - a.t0 : 0;
        if (a.steps > 0 && NWG == 2 && !a.pair) a_region ^= 1;
        a_step = 0;
        if (!(a_more = walk.next(a))) return true;
      }
      const int s = a_step++;
      const int q = a.pair ? (s & 1) : 0;                 // query tile
      const int rg = a.pair ? q : a_region;
      const bool q_first = a.pair ? s < 2 : s == 0, q_last = a.pair ? s >= a.steps - 2 : s == a.steps - 1;
      const long long i = 2 * (a_kv + (a.pair ? s >> 1 : s));
      const int st = (int)(i % NS), sb = (int)(a_total & 1);
      if (q_first) {
        if (!mbar_wait(bar(L::BAR_Q_FULL + rg), q_use[rg] & 1, wctx)) return false;
        ++q_use[rg];
      }
      if (!mbar_wait(bar(L::BAR_KV_FULL + st), (uint32_t)(i / NS) & 1u, wctx)) return false;
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        mma_ss(tmem + L::T_S(sb), sdesc_add(dQ0, rg * L::QTILE + (k / 4) * L::QCHUNK + (k % 4) * 32),
               sdesc_add(dK0, st * L::SLOT + (k / 4) * L::CHUNK + (k % 4) * 32), idesc_qk, k > 0 ? 1u : 0u, leader);
      }
      mma_commit(bar(L::BAR_S_FULL + sb), leader);
      if (!a.pair || q == 1) mma_commit(bar(L::BAR_KV_EMPTY + st), leader);
      if (q_last) mma_commit(bar(L::BAR_Q_EMPTY + rg), leader);
      ++a_total;
      return true;
    };
    ok = issue_s() && issue_s();
    Walk<D> pv_walk(p, start);
    long long kv = 0, total = 0;
    int o_use[2] = {0, 0}, p_cnt[2] = {0, 0};
    while (ok && pv_walk.next(sg)) {
      bool o_begun[2] = {false, false};
      for (int s = 0; s < sg.steps && ok; ++s, ++total) {
        const int sb = (int)(total & 1), w = NWG == 2 ? sb : 0;
        const long long i = 2 * (kv + (sg.pair ? s >> 1 : s)) + 1;
        const int st = (int)(i % NS);
        if (!o_begun[w]) {  // the accumulator's last results have been read
          if (o_use[w] > 0 && !(ok = mbar_wait(bar(L::BAR_O_FREE + w), (o_use[w] - 1) & 1, wctx))) break;
          ++o_use[w];
        }
        if (!(ok = mbar_wait(bar(L::BAR_KV_FULL + st), (uint32_t)(i / NS) & 1u, wctx))) break;
        if (!(ok = mbar_wait(bar(L::BAR_P_FULL + sb), p_cnt[sb] & 1, wctx))) break;
        ++p_cnt[sb];
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < KT / 16; ++k) {
          mma_ts(tmem + L::T_O(w), tmem + L::T_S(sb) + k * 8, sdesc_add(dV0, st * L::SLOT + k * 2048), idesc_pv,
                 (o_begun[w] || k > 0) ? 1u : 0u, leader);
        }
        o_begun[w] = true;
        if (!sg.pair || (s & 1)) mma_commit(bar(L::BAR_KV_EMPTY + st), leader);
        if (NWG == 1) mma_commit(bar(L::BAR_PV_DONE), leader);
        if (s == sg.steps - 1 || (sg.pair && s == sg.steps - 2)) mma_commit(bar(L::BAR_O_FULL + w), leader);
        ok = issue_s();
      }
      kv += sg.t1 - sg.t0;
    }
    mma_commit(bar(L::BAR_MMA_DONE), leader);
    drain_wait(bar(L::BAR_MMA_DONE), 0);
  } else if (warp < 4) {
    if constexpr (NWG == 2) regs_dec<kRegsLow>();
  } else {
    // ===================================================== softmax
    if constexpr (NWG == 2) regs_inc<kRegsHigh>();
    const int w = (warp - 4) >> 2;
    const int wq = warp & 3;
    const int row = wq * 32 + lane;
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    float2* stat = reinterpret_cast<float2*>(gbase + L::OFF_STAT);
    bool ok = true;
    long long kv = 0, total = 0;  // key tiles and steps of earlier segments
    int s_cnt[2] = {0, 0};        // steps in each S buffer
    int o_cnt = 0;                // segments that this warpgroup ended
    int stat_cnt = 0;             // statistics handed over (by either warpgroup)
    while (ok && walk.next(sg)) {
      const int p0 = (int)(total & 1);
      const int s_first = NWG == 2 ? (w ^ p0) : 0;
      const int s_by = NWG == 2 ? 2 : 1;
      const int tile_q = sg.pair ? s_first : 0;  // this warpgroup's query tile
      // rows of the tile, and this row's sequence or token
      int live;
      if (sg.own)
        live = min(128, p.R - sg.rc * ITEM - tile_q * 128);
      else
        live = min(p.seqs, p.B - sg.b - tile_q * p.seqs) * p.R;
      const bool warp_live = wq * 32 < live;
      bool counts = row < live;  // rows of a sequence that is not there may hold anything
      if (counts && !sg.own) counts = p.lens[sg.b + tile_q * p.seqs + row / p.R] >= 0;
      int own_lim = sg.visible;
      if (sg.own && p.causal) own_lim = sg.len - p.T + (sg.rc * ITEM + tile_q * 128 + row) % p.T + 1;
      float m = -INFINITY, l = 0.f;
      bool mine = false;
      for (int s = s_first; s < sg.steps; s += s_by) {
        const int sb = NWG == 2 ? w : (int)((total + s) & 1);
        const int kt = sg.pair ? s >> 1 : s;
        const TileInfo x = tile_info<KT>(p, sg, sg.t0 + kt);
        if (x.n < KT && (!sg.pair || s_first == 0)) {
          // the tile ends behind the last token: rows x.n .. of V are whatever was there before
          const long long i = 2 * (kv + kt) + 1;
          const int st = (int)(i % NS);
          if (!(ok = mbar_wait(bar(L::BAR_KV_FULL + st), (uint32_t)(i / NS) & 1u, wctx))) break;
          const int n16 = (KT - x.n) * 8;  // 16-byte units per chunk: whole rows, so the swizzle does not matter
          for (int c = 0; c < L::KCH; ++c)
            for (int z = (int)threadIdx.x & 127; z < n16; z += 128)
              *reinterpret_cast<uint4*>(gbase + L::OFF_KV + st * L::SLOT + c * L::CHUNK + x.n * 128 + z * 16) =
                  make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
        }
        if (!(ok = mbar_wait(bar(L::BAR_S_FULL + sb), s_cnt[sb] & 1, wctx))) break;
        ++s_cnt[sb];
        tc_fence_after();
        if (warp_live) {
          const int lim = x.pre ? x.n : min(x.n, own_lim - x.k0);
          ok = softmax_step<D, BF>(tmem + lanes + L::T_S(sb), tmem + lanes + L::T_O(w), p.scale_log2, lim, !mine, m, l,
                                   [&]() -> bool {
                                     // one accumulator: the previous step's product may still run
                                     if constexpr (NWG == 1)
                                       return mbar_wait(bar(L::BAR_PV_DONE), (uint32_t)(total + s - 1) & 1u, wctx);
                                     return true;
                                   });
          if (!ok) break;
          // weights are at most 2^8: a sum that is no finite number came from a non-finite score
          // (a wrong page may be the reason, and that report stays)
          if (counts && !(l <= 3.0e38f)) atomicCAS(p.err, kDevOk, kDevRange);
          tmem_wait_st();
        }
        mine = true;
        tc_fence_before();
        mbar_arrive(bar(L::BAR_P_FULL + sb));
      }
      total += sg.steps;
      kv += sg.t1 - sg.t0;
      if (!ok) break;
      if (!mine) continue;
      // ---- the end of a segment.  Two tiles: each warpgroup has its own rows.  One tile: the
      // warpgroup of the last step joins the other's m, l (through shared memory) and O.
      const bool other = NWG == 2 && !sg.pair && sg.steps > 1;
      const bool ends = sg.pair || NWG == 1 || ((int)(total - 1) & 1) == w;
      if (other) {
        if (!ends) {
          if (stat_cnt > 0 && !(ok = mbar_wait(bar(L::BAR_STAT_EMPTY), (stat_cnt - 1) & 1, wctx))) break;
          stat[row] = make_float2(m, l);
          mbar_arrive(bar(L::BAR_STAT_FULL));
          ++stat_cnt;
          continue;
        }
        if (!(ok = mbar_wait(bar(L::BAR_STAT_FULL), stat_cnt & 1, wctx))) break;
        ++stat_cnt;
      }
      float2 theirs = make_float2(-INFINITY, 0.f);
      if (other) {
        theirs = stat[row];
        mbar_arrive(bar(L::BAR_STAT_EMPTY));
      }
      if (!(ok = mbar_wait(bar(L::BAR_O_FULL + w), o_cnt & 1, wctx))) break;
      ++o_cnt;
      tc_fence_after();
      const float M = fmaxf(m, theirs.x);
      float ca = M == -INFINITY ? 0.f : ex2_approx(m - M);
      float cb = M == -INFINITY ? 0.f : ex2_approx(theirs.x - M);
      const float sum = ca * l + cb * theirs.y;
      const bool whole = sg.t0 == 0 && sg.t1 == sg.nt;
      const bool direct = whole && sg.own && (!p.packed || p.prefix_len == 0);
      const long long item = sg.own ? ((long long)sg.b * p.n_rc + sg.rc) * p.H_kv + sg.hk
                                    : (long long)sg.hk * p.n_groups + sg.b / (p.seqs * NWG);
      const long long items = sg.own ? (p.packed ? (long long)p.B * p.n_rc * p.H_kv : 0) : (long long)p.n_groups * p.H_kv;
      const int part = sg.own ? p.ctas - 1 - (int)blockIdx.x : (int)blockIdx.x;
      const long long slot = whole ? item : items + 2 * part + (sg.t0 == 0 ? 1 : 0);
      const int slot_rows = sg.own ? min(p.R, ITEM) : ITEM;
      const int in_slot = tile_q * 128 + wq * 32;  // first row of this warp in the slot
      const long long out_row = ((long long)sg.b * p.H_kv + sg.hk) * p.R + sg.rc * ITEM + in_slot;
      if (sg.own && sg.t0 == 0 && tile_q == 0 && row == 0) {
        // for the joining kernel: which parts of the line hold the item
        int last = part;
        if (!whole) {  // the item's last unit is nt - t1 units behind this part
          const int parts = line_parts(p, start.total);
          last = part_of(start.total, parts, part_begin(start.total, parts, part + 1) + (sg.nt - sg.t1) - 1);
        }
        p.seg[item] = make_int2(part, last);
      }
      const int left = live - wq * 32;  // live rows of this warp
      if (direct) {
        const float inv = sum > 0.f ? 1.0f / sum : 0.f;
        ca *= inv;
        cb *= inv;
      }
      const uint32_t tO = tmem + lanes + L::T_O(w), tO2 = tmem + lanes + L::T_O(w ^ 1);
      auto load = [&](int c, uint32_t (&u)[32]) {  // 32 columns of the joined O
        tmem_ld32(tO + 32 * c, u);
        if (other) {
          uint32_t v[32];
          tmem_ld32(tO2 + 32 * c, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i)
            u[i] = __float_as_uint(fmaf(ca, __uint_as_float(u[i]), cb * __uint_as_float(v[i])));
        } else {
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(ca * __uint_as_float(u[i]));
        }
        if (c == D / 32 - 1) {  // everything read
          tc_fence_before();
          mbar_arrive(bar(L::BAR_O_FREE + w));
          if (other) mbar_arrive(bar(L::BAR_O_FREE + (w ^ 1)));
        }
      };
      if (direct) {
        uint8_t* dst = static_cast<uint8_t*>(p.o) + out_row * (2 * D);
#pragma unroll 1
        for (int c = 0; c < D / 64; ++c) {
          uint4 a[8];
          uint32_t u[32];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            load(2 * c + h, u);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              auto at = [&](int k) { return __uint_as_float(u[8 * i + k]); };
              // a row that saw nothing has P = 0 and an accumulator of zeros
              a[4 * h + i] = make_uint4(pack16<BF>(at(0), at(1)), pack16<BF>(at(2), at(3)), pack16<BF>(at(4), at(5)),
                                        pack16<BF>(at(6), at(7)));
            }
          }
          warp_store_rows_128b(a, dst + c * 128, 2 * D, 0, left);
        }
        if (p.lse != nullptr && lane < left)
          p.lse[out_row + lane] = sum > 0.f ? (M + __log2f(sum)) * 0.69314718055994531f : -INFINITY;
      } else {
        const long long srow = slot * slot_rows + in_slot;
        float* part = (sg.own ? p.own_o : p.pre_o) + srow * D;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t u[32];
          load(c, u);
          uint4 a[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) a[i] = make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
          warp_store_rows_128b(a, reinterpret_cast<uint8_t*>(part) + c * 128, 4 * D, 0, left);
        }
        if (lane < left) (sg.own ? p.own_ml : p.pre_ml)[srow + lane] = make_float2(M, sum);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------- joining the parts
// One warp per query row.  Parts of the own keys, then of the prefix, in the order of their lines.
template <int D, bool BF>
__global__ void __launch_bounds__(256) fa_paged_join_kernel(const PagedParams p) {
  constexpr int NWG = PLayout<D>::NWG, KT = PLayout<D>::KT, ITEM = 128 * NWG;
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);  // (b * H + h) * T + t
  if (row >= (long long)p.B * p.H * p.T) return;
  const long long bk = row / p.R;  // b * H_kv + hk
  const int r = (int)(row - bk * p.R), b = (int)(bk / p.H_kv), hk = (int)(bk - (long long)b * p.H_kv);
  const int len = own_len(p, b);
  if (len < 0) return;
  const int rc = r / ITEM;
  const int nt = own_tiles<KT>(p, len, own_visible<ITEM>(p, len, rc));
  const bool pre = p.packed && p.prefix_len > 0;
  const long long item = ((long long)b * p.n_rc + rc) * p.H_kv + hk;
  int2 own = make_int2(0, -1), pc = make_int2(0, -1);
  if (nt > 0) {
    own = p.seg[item];
    if (own.x == own.y && !pre) return;  // written at once
  }
  long long pre_item = 0, pre_row = 0;
  if (pre) {
    const int per = p.seqs * NWG, g = b / per, in = b - g * per;
    pre_item = (long long)hk * p.n_groups + g;
    pre_row = (in / p.seqs) * 128 + (in % p.seqs) * p.R + r;
    const long long n = (long long)p.n_groups * p.H_kv * p.pre_tiles, u = pre_item * p.pre_tiles;
    const int parts = line_parts(p, n);
    pc.x = part_of(n, parts, u);
    pc.y = part_of(n, parts, u + p.pre_tiles - 1);
  }
  const int n_own = own.y - own.x + 1, n = n_own + pc.y - pc.x + 1;
  const long long own_items = p.packed ? (long long)p.B * p.n_rc * p.H_kv : 0;
  const long long pre_items = (long long)p.n_groups * p.H_kv;
  // where part i's row lies, counted in rows of its array
  auto at = [&](int i) -> long long {
    const bool o = i < n_own;
    const int2 c = o ? own : pc;
    const int part = c.x + (o ? i : i - n_own);
    const long long slot = c.x == c.y ? (o ? item : pre_item)
                                      : (o ? own_items : pre_items) + 2 * part + (part == c.x ? 1 : 0);
    return o ? slot * min(p.R, ITEM) + (r - rc * ITEM) : slot * ITEM + pre_row;
  };
  float M = -INFINITY, L = 0.f, o[E];
#pragma unroll
  for (int i = 0; i < E; ++i) o[i] = 0.f;
  for (int i0 = 0; i0 < n; i0 += 32) {
    float2 ml = make_float2(-INFINITY, 0.f);
    long long where = 0;
    if (i0 + lane < n) {
      where = at(i0 + lane);
      ml = (i0 + lane < n_own ? p.own_ml : p.pre_ml)[where];
    }
    float m = ml.x;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float mn = fmaxf(M, m);
    const float a = mn == -INFINITY ? 0.f : ex2_approx(M - mn);
    const float c = mn == -INFINITY ? 0.f : ex2_approx(ml.x - mn);
    float s = c * ml.y;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    L = fmaf(L, a, s);
    M = mn;
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] *= a;
    const int m32 = min(32, n - i0);
    for (int k = 0; k < m32; ++k) {
      const float ck = __shfl_sync(0xffffffffu, c, k);
      const long long wk = __shfl_sync(0xffffffffu, where, k);
      const float* src = (i0 + k < n_own ? p.own_o : p.pre_o) + wk * D + lane * E;
#pragma unroll
      for (int i = 0; i < E; i += 2) {
        const float2 v = *reinterpret_cast<const float2*>(src + i);
        o[i] = fmaf(ck, v.x, o[i]);
        o[i + 1] = fmaf(ck, v.y, o[i + 1]);
      }
    }
  }
  const float inv = L > 0.f ? 1.0f / L : 0.f;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.o) + (row * D + lane * E) * 2);
#pragma unroll
  for (int i = 0; i < E; i += 2) dst[i / 2] = pack16<BF>(o[i] * inv, o[i + 1] * inv);
  if (lane == 0 && p.lse != nullptr)
    p.lse[row] = L > 0.f ? (M + __log2f(L)) * 0.69314718055994531f : -INFINITY;
}

template <int D, bool BF>
cudaError_t launch(const PagedMaps& maps, const PagedParams& p, cudaStream_t s) {
  using L = PLayout<D>;
  auto kernel = fa_paged_attn_sm100_kernel<D, BF>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM_ALLOC);
  if (e != cudaSuccess) return e;
  kernel<<<p.ctas, L::THREADS, L::SMEM_ALLOC, s>>>(maps, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const long long rows = (long long)p.B * p.H * p.T;
  fa_paged_join_kernel<D, BF><<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(p);
  return cudaGetLastError();
}

template <bool BF>
cudaError_t launch(const PagedMaps& maps, const PagedParams& p, int d, cudaStream_t s) {
  return d == 64 ? launch<64, BF>(maps, p, s) : d == 128 ? launch<128, BF>(maps, p, s) : launch<256, BF>(maps, p, s);
}

}  // namespace

cudaError_t launch_paged_attn(const PagedMaps& maps, const PagedParams& p, int d, int dtype, cudaStream_t s) {
  return dtype == FA_BF16 ? launch<true>(maps, p, d, s) : launch<false>(maps, p, d, s);
}

}  // namespace fa
