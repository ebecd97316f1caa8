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
// Split.  A unit is one item and one tile of 128 keys (64 in the dense form at d = 256).  The units of
// all own items are one line, cut into equal parts for the persistent CTAs (one per multiprocessor),
// and so are those of the prefix items; a CTA walks its part of both lines.  So ragged lengths load
// all multiprocessors equally, without the host knowing them: every CTA adds up the lengths itself.
// A part that covers an item only partly leaves (m, l, O) in the workspace, and a second kernel joins
// the parts of each row in the order of the line (the same on every run).  Half of the CTAs walk the
// own line first: own items wait for memory (each key is used for R rows only), prefix items for the
// tensor core, and the two overlap across the device.  The halves are whole pairs of neighbouring
// multiprocessors (by smid): two neighbours in different code slow each other down by fetching
// instructions (128 sequences over a prefix of 32785 tokens, when this was chosen: 150 us with neighbours
// in different lines, 113 us so, 117 us with the prefix first everywhere).
//
// Two forms of a tile's products:
//   dense  S = Q K^T and O += P V with the query rows as the 128 rows of the product, for items of
//          more than 32 rows: two softmax warpgroups, one thread per row, take the steps in turn.
//   few    S^T = K Q^T and O^T += V^T P^T with the keys, then the columns of V, as the 128 rows and
//          the (up to 32) query rows as columns.  One thread per key then has one weight per query
//          row to compute instead of 128, all four warps work, and the rows of O^T are the elements
//          of o that are stored side by side.  With the dense form a step of a few rows took 2500
//          cycles (one warp's 128 exponentials) and its epilogue 2700, where a tile's share of the
//          memory bandwidth is 1400 (d = 64) or 2800.
// In both, warp 0 looks up pages and streams Q and K tiles with TMA, warp 2 V tiles, into one ring (a
// lane issues the box of a piece of a page; two warps, because a box costs its issuer some 70
// cycles and 8-token pages make 32 of them per tile), and warp 1 issues the tensor-core products, S
// of a step two steps ahead of its P V, across items.  Warp 3 walks the lines and hands the others what
// they need to know of each segment through shared memory: code that every role runs once per
// segment is code that none of them finds in the instruction cache (with a walk in each role,
// segments of one tile took 8000 cycles).
//
// Measured on B200 (bf16, 32 query and 8 key/value heads, d = 128): 37 sequences of 1 to 16384 own tokens,
// 1.24 GB of keys and values, 195 us (6.4 TB/s, 97 % of the measured copy rate), sequences of equal
// length (16384) 6.9 TB/s; the dense form against a prefix of 32785 tokens alone 256 us or 1.08 PFLOP/s for
// 512 sequences (66 % of the measured matrix rate: a step's chain of S, softmax and P V, two of which
// overlap, bounds it) and 85 us or 0.81 for 128, where a fixed 25 us (launch, code that the instruction
// caches do not hold yet, cut items, joining) counts; 128 sequences of 1 to 512 own tokens behind that
// prefix 114 us.
//
// What lies behind a sequence's last token in a page never enters: its scores are masked, and the rows of
// the V tile are set to zero in shared memory (0 x NaN would be NaN).  P is rounded to the 16-bit
// type for the second product; sums (of the weights before that rounding), maxima and O are fp32.
// Weights are 2^(s - m + kShift), where the running maximum m may lag the true one by kLag.  bf16 has
// fp32's exponents: kShift = 0, kLag = 8.  fp16 ends at 2^16 and rounds what is below 2^-25 to 0, which
// over 10^5 keys may be some thousandths of a row's weight: kShift = 7 moves that to 2^-32, and kLag = 4
// leaves 2^5 for the rounding of s - m where scores are large (below 2^27).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <atomic>

#include "paged.h"
#include "sm100.cuh"

namespace fa {
namespace {

constexpr int kThreads = 384;  // warp 0: Q, K; 1: products; 2: V; 3: schedule; 4-7 and 8-11: softmax
// registers: the first four warps give theirs to the two softmax warpgroups
constexpr uint32_t kRegsLaunch = 168, kRegsLow = 88, kRegsHigh = 208;
static_assert(kRegsLow + 2 * kRegsHigh <= 3 * kRegsLaunch, "register split exceeds the launch budget");

// Shared memory and tensor memory of the dense form.
template <int D>
struct Dense {
  static constexpr int KT = D == 256 ? 64 : 128;     // keys per tile
  static constexpr int NWG = D == 256 ? 1 : 2;       // softmax warpgroups = O accumulators = query tiles
  static constexpr int KCH = D / 64;                 // 128-byte column chunks per row
  static constexpr int QCHUNK = 128 * 128;           // one chunk of a query tile
  static constexpr int QTILE = KCH * QCHUNK;
  static constexpr int CHUNK = KT * 128;             // one chunk of a K or V tile
  static constexpr int SLOT = KCH * CHUNK;
  static constexpr int NS = D == 64 ? 11 : 5;        // ring slots
  static constexpr int OFF_KV = NWG * QTILE;
  static constexpr int OFF_STAT = OFF_KV + NS * SLOT;  // float2[128]: a warpgroup's m and l for the other
  static constexpr int END = OFF_STAT + 1024;
  static constexpr int HALVES = KT / 64;               // P is handed over in parts of 64 keys
  // barriers
  static constexpr int Q_FULL = 0, Q_EMPTY = 2, S_FULL = 4, P_FULL = 6 /* [2][2] */, O_FULL = 10, O_FREE = 12;
  static constexpr int STAT_FULL = 14, STAT_EMPTY = 15, PV_DONE = 16, MMA_DONE = 17, KV_FULL = 18, KV_EMPTY = 18 + NS;
  static constexpr int NBAR = 18 + 2 * NS;
  static_assert(NS >= 4, "S of a step is issued two steps ahead: two K and two V tiles are held at once");
  static __host__ __device__ constexpr uint32_t T_S(int i) { return i * KT; }
  static __host__ __device__ constexpr uint32_t T_O(int i) { return 256 + i * D; }
  static_assert(2 * KT <= 256 && 256 + NWG * D <= 512, "tensor memory columns");
};

// The same of the few-rows form.  A ring slot holds 128 keys x up to 128 columns; a tile is 128 keys,
// at d = 64 256 keys (two per softmax thread: what a step costs apart from its keys, waits and
// barriers of some 1000 cycles, then falls on 64 KB of keys and values, as at d = 128).
template <int D>
struct Few {
  static constexpr int KPT = D == 64 ? 2 : 1;        // keys per thread
  static constexpr int KT = 128 * KPT;
  static constexpr int KCH = D / 64;
  static constexpr int PARTS_D = D == 256 ? 2 : 1;   // slots per K or V tile along the columns
  static constexpr int PARTS = PARTS_D * KPT;        // slots per K or V tile
  static constexpr int PCH = KCH / PARTS_D;          // chunks per slot
  static constexpr int CHUNK = 128 * 128;
  static constexpr int SLOT = PCH * CHUNK;
  static constexpr int NS = D == 64 ? 10 : 5;
  static constexpr int NQ = D == 256 ? 2 : 4;        // query buffers
  static constexpr int RCHUNK = kFewRows * 128;      // one chunk (64 columns or keys) of Q or P^T
  static constexpr int PBUF = 2 * KPT * RCHUNK;      // 32 rows x the tile's keys
  static constexpr int OFF_Q = NS * SLOT;
  static constexpr int OFF_P = OFF_Q + NQ * KCH * RCHUNK;  // [2]
  static constexpr int OFF_EX = OFF_P + 2 * PBUF;          // float[2 warpgroups][2][32][4]
  static constexpr int END = OFF_EX + 2048;
  // the product of d = 64 takes 128 columns of V: the second 64 are whatever follows the slot
  static_assert(D != 64 || OFF_Q + CHUNK <= END, "the last slot's neighbour is inside shared memory");
  static constexpr int Q_FULL = 0, Q_EMPTY = NQ, S_FULL = 2 * NQ, P_FULL = S_FULL + 4, P_EMPTY = P_FULL + 2;
  static constexpr int O_FULL = P_EMPTY + 2, O_FREE = O_FULL + 2, MMA_DONE = O_FREE + 2, KV_FULL = MMA_DONE + 1;
  static constexpr int KV_EMPTY = KV_FULL + NS, NBAR = KV_EMPTY + NS;
  static __host__ __device__ constexpr uint32_t T_S(int i, int h) { return (i * 2 + h) * kFewRows; }        // [4][2]
  static __host__ __device__ constexpr uint32_t T_O(int i, int h) { return 256 + (i * 2 + h) * kFewRows; }  // [2][2]
};

constexpr int cmax(int a, int b) { return a > b ? a : b; }
// One item, or the part of it that falls into a CTA's part of a line.
struct Seg {
  int valid, own, pair;  // pair: dense form, two query tiles
  int b, hk, row0;       // prefix: b is the first sequence of tile 0; own: row0 is the first row of the item
  int rows[2];           // rows of the query tiles (few form: of the item)
  int len, visible;      // own: the sequence's length, and its keys seen by some row
  int lead;              // key tiles below `lead` are the prefix's
  int t0, t1;            // key tiles
  int direct;            // the item is whole and nothing is to be joined: results go to o and lse
  uint8_t* o_dst;        // first row's result (16-bit) or partial result (fp32)
  void* ml_dst;          // first row's lse (float, or null), or its (maximum, sum)
};
constexpr int kSegRing = 4;
constexpr int kSegReaders = 11;  // warps that read each segment

template <int D>
struct Smem {
  static constexpr int OFF_BAR = cmax(Dense<D>::END, Few<D>::END);
  static constexpr int DENSE_BAR = 0, FEW_BAR = Dense<D>::NBAR, SEG_FULL = FEW_BAR + Few<D>::NBAR;
  static constexpr int SEG_EMPTY = SEG_FULL + kSegRing, NBAR = SEG_EMPTY + kSegRing;
  static constexpr int OFF_SEG = OFF_BAR + NBAR * 8;
  static constexpr int OFF_START = OFF_SEG + kSegRing * (int)sizeof(Seg);
  static constexpr int OFF_SCAN = OFF_START + 48;  // int[12]
  static constexpr int OFF_TMEM_SLOT = OFF_SCAN + 96;
  static constexpr int OFF_ABORT = OFF_TMEM_SLOT + 8;
  static constexpr int OFF_ISSUED = OFF_ABORT + 8;  // uint32[2]: ring index behind the last K and V slot asked for
  static constexpr int ALLOC = OFF_ISSUED + 8 + 1024;
  static_assert(ALLOC <= 232448, "shared memory per CTA");
};

// mbar_wait in as few instructions as it takes (the segments' code competes for the instruction
// cache): the same limit, on the low word of the timer, and an abort flag; the end of the phase puts
// that into the error word.  For whole warps: the answer is the same for all 32 threads, which go on
// together (to instructions that need all of them) or give up together.
struct Waits {
  uint32_t abort_flag;  // shared memory address
};
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, const Waits& w) {
  static_assert(kWaitLimitNs < (1ull << 32), "the limit fits the timer's low word");
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b32 t0, t1;\n\t"
      "mov.u32 %0, 1;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE;\n\t"
      "mov.u32 t0, %globaltimer_lo;\n\t"
      "AGAIN:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "@p bra DONE;\n\t"
      "ld.volatile.shared::cta.u32 t1, [%3];\n\t"
      "setp.ne.u32 p, t1, 0;\n\t"
      "@p bra FAIL;\n\t"
      "mov.u32 t1, %globaltimer_lo;\n\t"
      "sub.u32 t1, t1, t0;\n\t"
      "setp.lt.u32 p, t1, %4;\n\t"
      "@p bra AGAIN;\n\t"
      "st.volatile.shared::cta.u32 [%3], 1;\n\t"
      "FAIL:\n\t"
      "mov.u32 %0, 0;\n\t"
      "DONE:\n\t"
      "setp.ne.u32 p, %0, 0;\n\t"
      "vote.sync.all.pred p, p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(w.abort_flag), "n"((uint32_t)kWaitLimitNs)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (globaltimer_ns() - t0 > kWaitLimitNs) break;
  }
}

// After a phase in which a wait gave up: every K and V copy asked for has landed (or the bounded
// waits run out).  `asked[v]` is the ring index behind the last slot that the K (v = 0) or V warp asked
// for, `parts` slots make a tile; the last index of a slot tells its barrier's phase.
template <int NS>
__device__ __forceinline__ void drain_ring(uint32_t bar_full, int parts, const volatile uint32_t* asked) {
  for (uint32_t s = 0; s < NS; ++s) {
    int last = -1;
    for (int v = 0; v < 2; ++v)
      for (int k = (int)asked[v] - 1; k >= 0 && k >= (int)asked[v] - 4 * NS; --k)
        if ((uint32_t)k % NS == s && (k / parts & 1) == v) {
          last = max(last, k);
          break;
        }
    if (last >= 0) drain_wait(bar_full + 8u * s, (uint32_t)last / NS & 1u);
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

// N = 4, 8, 16 or 32 consecutive columns of this warp's 32 lanes.
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[N]) {
  static_assert(N == 4 || N == 8 || N == 16 || N == 32, "column counts in use");
  if constexpr (N == 32) {
    tmem_ld32(taddr, r);
  } else if constexpr (N == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  } else if constexpr (N == 4) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr));
  } else {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
  }
}
// Keeps every use of loaded registers behind the wait for them (the compiler knows of no tie between
// a load and the wait).
template <int N>
__device__ __forceinline__ void loaded(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[N]) {
  if constexpr (N == 32)
    tmem_st32(taddr, r);
  else if constexpr (N == 16)
    tmem_st16(taddr, r);
  else if constexpr (N == 8)
    tmem_st8(taddr, r);
  else
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3])
                 : "memory");
}

// Whether any of the 128 threads of a warpgroup says so; a barrier among them as well.
__device__ __forceinline__ bool group_any(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void group_sync(int id) { named_bar_sync((uint32_t)id, 128); }

__device__ __forceinline__ void st_global_32b(void* dst, const uint32_t* v) {  // 32-byte aligned
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

__device__ __forceinline__ void st_shared_u16(uint32_t addr, uint16_t x) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(x) : "memory");
}

template <bool BF>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
  return BF ? pack_bf16(a, b) : pack_f16(a, b);
}
template <bool BF>
__device__ __forceinline__ uint16_t round16(float a) {
  if constexpr (BF)
    return __bfloat16_as_ushort(__float2bfloat16_rn(a));
  else
    return __half_as_ushort(__float2half_rn(a));
}
// Natural logarithm of 2^m l: -inf for a row that sees no key, NaN where the keys that it sees have no sum.
__device__ __forceinline__ float log_sum(float m, float l, bool sees) {
  return l > 0.f ? (m + __log2f(l)) * 0.69314718055994531f : sees ? __int_as_float(0x7fffffff) : -INFINITY;
}
// A mean of finite fp16 values, off by the rounding of its weights (2^-11), may pass fp16's end: it is that end.
// (bf16's is as far as fp32's.)
template <bool BF>
__device__ __forceinline__ float to_range(float x) {
  if constexpr (BF) return x;
  return fabsf(x) < 65600.0f ? fminf(fmaxf(x, -65504.0f), 65504.0f) : x;
}
// Inputs that are not finite, scores and sums beyond fp32 all end in an output that is not finite (a row
// that sees keys divides by its sum even if that is 0 or NaN).  So outputs are looked at when they are
// written, before the rounding: `z` gathers 0 x, which is NaN for such an x.  A wrong page may be the reason
// of one, and that report stays.
__device__ __forceinline__ void not_finite(float& z, float x) { z = fmaf(x, 0.f, z); }
__device__ __forceinline__ void report_range(float z, int* err) {
  if (z != 0.f) atomicCAS(err, kDevOk, kDevRange);
}

template <bool BF>
constexpr float kShift = BF ? 0.0f : 7.0f;
template <bool BF>
constexpr float kLag = BF ? 8.0f : 4.0f;

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
__device__ __forceinline__ int own_tiles(const PagedParams& p, int len, int visible) {
  if (len < 0) return 0;
  return (p.packed ? 0 : p.pre_tiles) + ((visible + (1 << p.own_kt) - 1) >> p.own_kt);
}
// Length of an item on the line: kItemCost for its beginning and end, then its tiles.
__device__ __forceinline__ int item_units(int tiles) { return tiles > 0 ? tiles + kItemCost : 0; }

template <int ITEM>
__device__ int units_of(const PagedParams& p, int b) {
  const int len = own_len(p, b);
  int n = 0;
  for (int rc = 0; rc < p.n_rc; ++rc) n += item_units(own_tiles(p, len, own_visible<ITEM>(p, len, rc)));
  return n * p.H_kv;
}

// A line of n units (fewer than 2^31, which the host sees to) in `parts` parts, none of them empty: the
// first `more` have size + 1 units, the others `size`.  The own line's parts go to the CTAs in falling
// order, so that a short prefix line and a short own line fall to different CTAs.
struct Line {
  int parts, size, more;
  __device__ __forceinline__ Line(int n, int ctas) {
    parts = min(n, ctas);
    size = parts > 0 ? (int)((unsigned)n / (unsigned)parts) : 0;
    more = n - size * parts;
  }
  __device__ __forceinline__ int begin(int part) const { return part * size + min(part, more); }
  __device__ __forceinline__ int part_of(int u) const {  // the part that holds unit u
    const int lead = more * (size + 1);
    return u < lead ? (int)((unsigned)u / (unsigned)(size + 1)) : more + (int)((unsigned)(u - lead) / (unsigned)size);
  }
};

struct Start {  // where a CTA's part of the own line begins
  int total;          // units of the whole line
  int left;           // units of this CTA
  int b, rc, hk, at;  // item, and the unit inside it
};

// Walks a CTA's segments of one line or both.
template <int D>
struct Walk {
  static constexpr int NWG = Dense<D>::NWG, ITEM = 128 * NWG;
  const PagedParams& p;
  const Start& start;
  int pre_u, pre_end, own_left;
  int b, rc, hk, at;
  int cur_b, len;

  __device__ Walk(const PagedParams& p_, const Start& s, bool pre, bool own) : p(p_), start(s) {
    const Line line(pre ? p.n_groups * p.H_kv * p.pre_tiles : 0, p.ctas);
    const int c = blockIdx.x;
    pre_u = c < line.parts ? line.begin(c) : 0;
    pre_end = c < line.parts ? line.begin(c + 1) : 0;
    own_left = own ? s.left : 0;
    b = s.b;
    rc = s.rc;
    hk = s.hk;
    at = s.at;
    cur_b = -1;
    len = 0;
  }
  // Where the results go.
  __device__ void place(Seg& s, bool whole, int item, int items, int part, int item_rows, long long out_row) {
    s.direct = whole && s.own && (!p.packed || p.prefix_len == 0);
    if (s.direct) {
      s.o_dst = static_cast<uint8_t*>(p.o) + out_row * (2 * D);
      s.ml_dst = p.lse != nullptr ? p.lse + out_row : nullptr;
    } else {
      const long long row = (long long)(whole ? item : items + 2 * part + (s.t0 == 0 ? 1 : 0)) * item_rows;
      s.o_dst = reinterpret_cast<uint8_t*>((s.own ? p.own_o : p.pre_o) + row * D);
      s.ml_dst = (s.own ? p.own_ml : p.pre_ml) + row;
    }
  }
  __device__ bool next(Seg& s, bool own_first) {
    if (own_first && next_own(s)) return true;
    if (pre_u < pre_end) {
      const int item = (int)((unsigned)pre_u / (unsigned)p.pre_tiles);
      s.own = 0;
      s.hk = (int)((unsigned)item / (unsigned)p.n_groups);
      s.b = (item - s.hk * p.n_groups) * p.group_seqs;
      s.row0 = s.len = s.visible = 0;
      s.lead = p.pre_tiles;
      s.t0 = pre_u - item * p.pre_tiles;
      s.t1 = min(p.pre_tiles, s.t0 + (pre_end - pre_u));
      s.pair = p.group_seqs > p.seqs && s.b + p.seqs < p.B;
      s.rows[0] = min(p.seqs, p.B - s.b) * p.R;
      s.rows[1] = s.pair ? min(p.seqs, p.B - s.b - p.seqs) * p.R : 0;
      pre_u += s.t1 - s.t0;
      place(s, s.t0 == 0 && s.t1 == p.pre_tiles, item, p.n_groups * p.H_kv, blockIdx.x, p.pre_rows, 0);
      return true;
    }
    return next_own(s);
  }
  __device__ bool next_own(Seg& s) {
    while (b < p.B && own_left > 0) {
      if (cur_b != b) {
        len = own_len(p, b);
        cur_b = b;
      }
      const int vis = own_visible<ITEM>(p, len, rc);
      const int nt = own_tiles(p, len, vis);
      int t0 = 0, t1 = 0;
      if (nt > 0) {
        const int end = min(nt + kItemCost, at + own_left);
        t0 = max(0, at - kItemCost);
        t1 = max(0, end - kItemCost);
        own_left -= end - at;
      }
      at = 0;
      const int rc0 = rc;
      s.hk = hk;
      s.b = b;
      // past this item (a part that ends inside it has nothing left); an item without tiles has none
      // for the other heads either
      if (nt == 0 || ++hk == p.H_kv) {
        hk = 0;
        if (++rc == p.n_rc) {
          rc = 0;
          ++b;
        }
      }
      if (t1 > t0) {
        s.own = 1;
        s.row0 = rc0 * ITEM;
        s.rows[0] = min(128, p.R - s.row0);
        s.rows[1] = NWG == 2 ? max(0, min(128, p.R - s.row0 - 128)) : 0;
        s.pair = s.rows[1] > 0;
        s.len = len;
        s.visible = vis;
        s.lead = p.packed ? 0 : p.pre_tiles;
        s.t0 = t0;
        s.t1 = t1;
        const int part = p.ctas - 1 - (int)blockIdx.x;
        const int item = (s.b * p.n_rc + rc0) * p.H_kv + s.hk;
        place(s, t0 == 0 && t1 == nt, item, p.packed ? p.B * p.n_rc * p.H_kv : 0, part, min(p.R, ITEM),
              ((long long)s.b * p.H_kv + s.hk) * p.R + s.row0);
        if (t0 == 0 && threadIdx.x % 32 == 0) {  // for the joining kernel: which parts of the line hold the item
          int last = part;
          if (t1 < nt) {  // its last unit is nt - t1 units behind this part
            const Line line(start.total, p.ctas);
            last = line.part_of(line.begin(part + 1) + (nt - t1) - 1);
          }
          p.seg[item] = make_int2(part, last);
        }
        return true;
      }
    }
    own_left = 0;
    return false;
  }
};

// The segments' ring, as the readers see it: segment `no` of this CTA, copied out of shared memory.
struct SegRing {
  const Seg* ring;
  uint32_t full, empty;  // barriers
  uint32_t no;
  __device__ __forceinline__ bool next(Seg& s, const Waits& wctx) {
    const uint32_t slot = no % kSegRing;
    if (!wait_bar(full + 8u * slot, no / kSegRing & 1u, wctx)) return false;
    s = ring[slot];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(empty + 8u * slot);
    ++no;
    return s.valid != 0;
  }
};
// Warp 3: the segments of a phase, and one that says that there are no more.
template <int D>
__device__ __forceinline__ void schedule(const PagedParams& p, const Start& start, bool pre, bool own, bool own_first,
                                         Seg* ring, uint32_t full, uint32_t empty, uint32_t& no,
                                         volatile int* abort_flag, const Waits& wctx) {
  Walk<D> walk(p, start, pre, own);
  for (bool more = true; more; ++no) {
    Seg s;
    more = walk.next(s, own_first);
    s.valid = more;
    const uint32_t slot = no % kSegRing;
    if ((int)no + 1 == p.give_up) *abort_flag = 1;  // (self-test)
    if (no >= kSegRing && !wait_bar(empty + 8u * slot, (no / kSegRing - 1) & 1u, wctx)) return;
    if ((threadIdx.x & 31) == 0) {
      ring[slot] = s;
      mbar_arrive(full + 8u * slot);
    }
    __syncwarp();
  }
}

// Key tile `t` of a segment: whether it is the prefix's, its first token there and its tokens.
struct TileInfo {
  bool pre;
  int k0, n;
};
template <int KT>
__device__ __forceinline__ TileInfo tile_info(const PagedParams& p, const Seg& s, int t) {
  TileInfo x;
  x.pre = t < s.lead;
  x.k0 = (x.pre ? t : t - s.lead) * KT;
  x.n = min(KT, (x.pre ? p.prefix_len : s.visible) - x.k0);
  return x;
}

// The page of a tile's piece that starts at token `row0` of the tile.
__device__ __forceinline__ int look_up(const PagedParams& p, const Seg& s, const TileInfo& x, int row0) {
  const int none = max(p.num_pages, 1);  // one behind the last page: TMA reads zeros there
  if (row0 >= x.n) return none;
  const int e = (x.k0 + row0) >> p.page_shift;
  const int page = x.pre ? p.prefix_table[e] : p.table[(long long)s.b * p.table_stride + e];
  if (page >= 0 && page < p.num_pages) return page;
  atomicExch(p.err, kDevIndex);
  return none;
}

// Rows n .. of the keys of a V tile in shared memory set to zero (whole rows: the swizzle, which moves
// 16-byte units inside a row, does not matter), by the 128 threads of a warpgroup.
__device__ __forceinline__ void zero_rows(uint8_t* slot, int chunks, int chunk_bytes, int n) {
  const int units = (chunk_bytes - n * 128) / 16;
#pragma unroll 1
  for (int c = 0; c < chunks; ++c)
#pragma unroll 1
    for (int z = (int)threadIdx.x & 127; z < units; z += 128)
      *reinterpret_cast<uint4*>(slot + c * chunk_bytes + n * 128 + z * 16) = make_uint4(0, 0, 0, 0);
}

// ---------------------------------------------------------------------------- dense form: softmax step
// One step of a row: S from tensor memory, keys from `lim` on masked, running maximum, O rescaled
// when the maximum has moved by more than kLag, P back over S in parts of 64 keys (each announced on
// its barrier, so that P V starts while the next part is computed).  `ready` waits until O may be touched.
template <int D, bool BF, class Ready>
__device__ __forceinline__ bool dense_step(uint32_t tS, uint32_t tO, float sl2, int lim, bool first, float& m, float& l,
                                           uint32_t bar_p, Ready ready) {
  constexpr int KT = Dense<D>::KT;
  float x[KT];
  {
    uint32_t u[KT / 32][32];
#pragma unroll
    for (int c = 0; c < KT / 32; ++c) tmem_ld32(tS + 32 * c, u[c]);
    tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < KT / 32; ++c) loaded(u[c]);
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
  const float m_use = (m_new - m > kLag<BF>) ? m_new : m;
  const float alpha = (m_use == m) ? 1.0f : ex2_approx(m - m_use);  // 0 while nothing was visible before
  const float neg_m = m_use == -INFINITY ? 0.0f : kShift<BF> - m_use;  // nothing visible yet: every P is 0
  if (!first && __any_sync(0xffffffffu, alpha != 1.0f)) {
    if (!ready()) return false;
    tc_fence_after();
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      uint32_t u[32];
      tmem_ld32(tO + 32 * c, u);
      tmem_wait_ld();
      loaded(u);
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
    tmem_wait_st();
    tc_fence_before();
    mbar_arrive(bar_p + 8u * h);
  }
  float s0, s1, s2, s3;
  f2unpack(sa, s0, s1);
  f2unpack(sb, s2, s3);
  l = fmaf(l, alpha, (s0 + s1) + (s2 + s3));
  m = m_use;
  return true;
}

// ---------------------------------------------------------------------------- dense form
// Warps 0 - 3: copies and products.
template <int D, bool BF>
__device__ __forceinline__ void dense_feed(const PagedMaps& maps, const PagedParams& p, SegRing& segs, uint32_t base,
                                           uint32_t bars, uint32_t tmem, volatile uint32_t* asked_for,
                                           const Waits& wctx) {
  using L = Dense<D>;
  constexpr int KT = L::KT, NWG = L::NWG;
  constexpr uint32_t NS = L::NS;
  auto bar = [&](int i) -> uint32_t { return bars + 8u * i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Seg sg;

  if (warp == 0 || warp == 2) {
    // ===================================================== page lookup and TMA: Q and K, or V
    const int v = warp >> 1;
    const CUtensorMap* map = v ? &maps.v : &maps.k;
    const int per_chunk = KT / p.box_rows;  // boxes per column chunk of a tile
    const int chunk = lane / per_chunk, row0 = (lane - chunk * per_chunk) * p.box_rows;
    const bool has_box = chunk < L::KCH;
    const int page_mask = (1 << p.page_shift) - 1;
    uint32_t i = v, issued = 0;  // ring index of the next tile
    int q_count[2] = {0, 0}, region = 0;
    bool ok = true;
    while (ok && segs.next(sg, wctx)) {
      TileInfo x = tile_info<KT>(p, sg, sg.t0);
      int page = has_box ? look_up(p, sg, x, row0) : 0;
      if (v == 0) {
        // Q: one region for a single tile (the other one keeps the previous item's), both for two tiles
        for (int w = 0; w < (sg.pair ? 2 : 1); ++w) {
          const int rg = sg.pair ? w : region;
          if (q_count[rg] > 0 && !(ok = wait_bar(bar(L::Q_EMPTY + rg), (q_count[rg] - 1) & 1, wctx))) break;
          const int rows = min(p.R, 128) * (sg.own ? 1 : p.seqs);
          if (lane == 0) mbar_arrive_expect_tx(bar(L::Q_FULL + rg), (uint32_t)rows * 128u * L::KCH);
          __syncwarp();
          if (lane < L::KCH)
            tma_load_4d(base + rg * L::QTILE + lane * L::QCHUNK, sg.own ? &maps.q_own : &maps.q_pre, lane * 64,
                        sg.row0 + w * 128 * sg.own, sg.hk, sg.own ? sg.b : sg.b + w * p.seqs,
                        bar(L::Q_FULL + rg));
          ++q_count[rg];
        }
        if (!ok) break;
        if (NWG == 2 && !sg.pair) region ^= 1;
      }
      for (int t = sg.t0; t < sg.t1; ++t, i += 2) {
        const TileInfo y = x;
        const int cur = page;
        if (t + 1 < sg.t1) {
          x = tile_info<KT>(p, sg, t + 1);
          if (has_box) page = look_up(p, sg, x, row0);
        }
        const uint32_t st = i % NS;
        if (!(ok = wait_bar(bar(L::KV_EMPTY + st), (i / NS & 1u) ^ 1u, wctx))) break;
        const uint32_t boxes = (y.n + p.box_rows - 1) / p.box_rows;
        if (lane == 0) mbar_arrive_expect_tx(bar(L::KV_FULL + st), boxes * p.box_rows * 128u * L::KCH);
        __syncwarp();
        if (has_box && row0 < y.n)
          tma_load_4d(base + L::OFF_KV + st * L::SLOT + chunk * L::CHUNK + row0 * 128, map, chunk * 64,
                      (y.k0 + row0) & page_mask, sg.hk, cur, bar(L::KV_FULL + st));
        issued = i + 1;
      }
    }
    if (lane == 0) asked_for[v] = issued;
    // the copies of Q have landed before the phase ends (at once, unless a wait gave up)
    for (int rg = 0; rg < 2; ++rg)
      if (q_count[rg] > 0) drain_wait(bar(L::Q_FULL + rg), (q_count[rg] - 1) & 1);
  } else if (warp == 1) {
    // ===================================================== products
    const uint32_t leader = elect_one();
    constexpr uint32_t idesc_qk = make_idesc(128, KT, BF, false, false);
    constexpr uint32_t idesc_pv = make_idesc(128, D, BF, false, true);
    const uint64_t dQ0 = make_sdesc_sw128(base, 16, 1024);
    const uint64_t dK0 = make_sdesc_sw128(base + L::OFF_KV, 16, 1024);
    const uint64_t dV0 = make_sdesc_sw128(base + L::OFF_KV, L::CHUNK, 1024);
    bool ok = true;
    // what the P V of a step has to know, kept from its S, two steps earlier
    struct Step {
      bool valid, first, last_use, ends;
      uint32_t i;  // ring index of the V tile
    };
    int n_steps = 0, s = 0, region = 0, q_use[2] = {0, 0};
    uint32_t seg_i = 0, s_total = 0;  // ring index of the segment's first K tile; steps so far
    bool more = true, have = false;
    auto issue_s = [&]() -> Step {
      Step f{};
      if (!more) return f;
      if (s == n_steps) {
        if (have) {
          seg_i += 2 * (sg.t1 - sg.t0);
          if (NWG == 2 && !sg.pair) region ^= 1;
        }
        if (!(more = segs.next(sg, wctx))) return f;
        have = true;
        s = 0;
        n_steps = (sg.t1 - sg.t0) << (sg.pair ? 1 : 0);
      }
      const int q = sg.pair ? (s & 1) : 0;  // query tile
      const int rg = sg.pair ? q : region, per = sg.pair ? 2 : 1;
      const uint32_t i = seg_i + 2u * (uint32_t)(sg.pair ? s >> 1 : s), st = i % NS, sb = s_total & 1u;
      if (s < per) {
        if (!(ok = wait_bar(bar(L::Q_FULL + rg), q_use[rg] & 1, wctx))) return f;
        ++q_use[rg];
      }
      if (!(ok = wait_bar(bar(L::KV_FULL + st), i / NS & 1u, wctx))) return f;
      tc_fence_after();
      const uint64_t dq = sdesc_add(dQ0, rg * L::QTILE), dk = sdesc_add(dK0, st * L::SLOT);
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        mma_ss(tmem + L::T_S(sb), sdesc_add(dq, (k / 4) * L::QCHUNK + (k % 4) * 32),
               sdesc_add(dk, (k / 4) * L::CHUNK + (k % 4) * 32), idesc_qk, k > 0 ? 1u : 0u, leader);
      mma_commit(bar(L::S_FULL + sb), leader);
      if (q == per - 1) mma_commit(bar(L::KV_EMPTY + st), leader);
      if (s >= n_steps - per) mma_commit(bar(L::Q_EMPTY + rg), leader);
      f.valid = true;
      f.first = s < NWG;  // this accumulator's first product of the segment
      f.last_use = q == per - 1;
      f.ends = s >= n_steps - per;
      f.i = i + 1;
      ++s;
      ++s_total;
      return f;
    };
    Step f0 = issue_s();
    Step f1{};
    if (ok) f1 = issue_s();
    int o_use[2] = {0, 0};
    for (uint32_t total = 0; ok && f0.valid; ++total) {
      const uint32_t sb = total & 1u, w = NWG == 2 ? sb : 0, st = f0.i % NS;
      if (f0.first) {  // the accumulator's last results have been read
        if (o_use[w] > 0 && !(ok = wait_bar(bar(L::O_FREE + w), (o_use[w] - 1) & 1, wctx))) break;
        ++o_use[w];
      }
      if (!(ok = wait_bar(bar(L::KV_FULL + st), f0.i / NS & 1u, wctx))) break;
      const uint64_t dv = sdesc_add(dV0, st * L::SLOT);
#pragma unroll
      for (int h = 0; h < L::HALVES; ++h) {
        if (!(ok = wait_bar(bar(L::P_FULL + 2 * sb + h), total / 2 & 1u, wctx))) break;
        tc_fence_after();
#pragma unroll
        for (int k = 4 * h; k < 4 * h + 4; ++k)
          mma_ts(tmem + L::T_O(w), tmem + L::T_S(sb) + k * 8, sdesc_add(dv, k * 2048), idesc_pv,
                 (!f0.first || k > 0) ? 1u : 0u, leader);
      }
      if (!ok) break;
      if (f0.last_use) mma_commit(bar(L::KV_EMPTY + st), leader);
      if (NWG == 1) mma_commit(bar(L::PV_DONE), leader);
      if (f0.ends) mma_commit(bar(L::O_FULL + w), leader);
      f0 = f1;
      f1 = issue_s();
    }
    mma_commit(bar(L::MMA_DONE), leader);
    drain_wait(bar(L::MMA_DONE), 0);
  }
}

// Warps 4 - 11: softmax.
template <int D, bool BF>
__device__ __forceinline__ void dense_softmax(const PagedParams& p, SegRing& segs, uint8_t* gbase, uint32_t bars,
                                              uint32_t tmem, const Waits& wctx) {
  using L = Dense<D>;
  constexpr int KT = L::KT, NWG = L::NWG;
  constexpr uint32_t NS = L::NS;
  auto bar = [&](int i) -> uint32_t { return bars + 8u * i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w = (warp - 4) >> 2;
  Seg sg;
  if (w >= NWG) {  // d = 256: one warpgroup only, the other reads along
    while (segs.next(sg, wctx)) {
    }
  } else {
    const int wq = warp & 3;
    const int row = wq * 32 + lane;
    const uint32_t lanes = (uint32_t)(wq * 32) << 16;
    float2* stat = reinterpret_cast<float2*>(gbase + L::OFF_STAT);
    bool ok = true;
    uint32_t kv = 0, total = 0;  // key tiles and steps of earlier segments
    int o_cnt = 0;               // segments that this warpgroup ended
    int stat_cnt = 0;            // statistics handed over (by either warpgroup)
    while (ok && segs.next(sg, wctx)) {
      const int steps = (sg.t1 - sg.t0) << (sg.pair ? 1 : 0);
      const int s_first = NWG == 2 ? (w ^ (int)(total & 1u)) : 0;
      const int tile_q = sg.pair ? s_first : 0;  // this warpgroup's query tile
      // rows of the tile
      const int live = tile_q ? sg.rows[1] : sg.rows[0];
      const bool warp_live = wq * 32 < live;
      int own_lim = sg.visible;
      if (sg.own && p.causal) own_lim = sg.len - p.T + (sg.row0 + tile_q * 128 + row) % p.T + 1;
      float m = -INFINITY, l = 0.f;
      bool mine = false;
      for (int s = s_first; s < steps; s += NWG) {
        const uint32_t n = total + s, sb = n & 1u;
        const int kt = sg.pair ? s >> 1 : s;
        const TileInfo x = tile_info<KT>(p, sg, sg.t0 + kt);
        if (x.n < KT && (!sg.pair || s_first == 0)) {
          // the tile ends behind the last token: rows x.n .. of V are whatever was there before
          const uint32_t i = 2 * (kv + kt) + 1, st = i % NS;
          if (!(ok = wait_bar(bar(L::KV_FULL + st), i / NS & 1u, wctx))) break;
          zero_rows(gbase + L::OFF_KV + st * L::SLOT, L::KCH, L::CHUNK, x.n);
          fence_proxy_async_smem();
        }
        if (!(ok = wait_bar(bar(L::S_FULL + sb), n / 2 & 1u, wctx))) break;
        tc_fence_after();
        const uint32_t bar_p = bar(L::P_FULL + 2 * sb);
        if (warp_live) {
          const int lim = x.pre ? x.n : min(x.n, own_lim - x.k0);
          ok = dense_step<D, BF>(tmem + lanes + L::T_S(sb), tmem + lanes + L::T_O(w), p.scale_log2, lim, !mine, m, l,
                                 bar_p, [&]() -> bool {
                                   // one accumulator: the previous step's product may still run
                                   if constexpr (NWG == 1) return wait_bar(bar(L::PV_DONE), (n - 1) & 1u, wctx);
                                   return true;
                                 });
          if (!ok) break;
        } else {
          for (int h = 0; h < L::HALVES; ++h) mbar_arrive(bar_p + 8u * h);
        }
        mine = true;
      }
      total += steps;
      kv += sg.t1 - sg.t0;
      if (!ok) break;
      if (!mine) continue;
      // ---- the end of a segment.  Two tiles: each warpgroup has its own rows.  One tile: the
      // warpgroup of the last step joins the other's m, l (through shared memory) and O.
      const bool other = NWG == 2 && !sg.pair && steps > 1;
      float2 theirs = make_float2(-INFINITY, 0.f);
      if (other) {
        if (((total - 1) & 1u) != (uint32_t)w) {
          if (stat_cnt > 0 && !(ok = wait_bar(bar(L::STAT_EMPTY), (stat_cnt - 1) & 1, wctx))) break;
          stat[row] = make_float2(m, l);
          mbar_arrive(bar(L::STAT_FULL));
          ++stat_cnt;
          continue;
        }
        if (!(ok = wait_bar(bar(L::STAT_FULL), stat_cnt & 1, wctx))) break;
        ++stat_cnt;
        theirs = stat[row];
        mbar_arrive(bar(L::STAT_EMPTY));
      }
      if (!(ok = wait_bar(bar(L::O_FULL + w), o_cnt & 1, wctx))) break;
      ++o_cnt;
      tc_fence_after();
      const float M = fmaxf(m, theirs.x);
      float ca = M == -INFINITY ? 0.f : ex2_approx(m - M);
      float cb = M == -INFINITY ? 0.f : ex2_approx(theirs.x - M);
      const float sum = ca * l + cb * theirs.y;
      const bool sees = sg.lead > 0 || own_lim > 0;
      float z = 0.f;
      if (sg.direct) {
        const float inv = sees ? 1.0f / sum : 0.f;
        ca *= inv;
        cb *= inv;
      }
      const bool write = row < live;
      const int irow = tile_q * 128 + row;  // row of the item
      const uint32_t tO = tmem + lanes + L::T_O(w), tO2 = tmem + lanes + L::T_O(w ^ 1);
      uint8_t* dst = sg.o_dst + (size_t)irow * (sg.direct ? 2 * D : 4 * D);
      if (warp_live) {
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t u[32];
          tmem_ld32(tO + 32 * c, u);
          if (other) {
            uint32_t v[32];
            tmem_ld32(tO2 + 32 * c, v);
            tmem_wait_ld();
            loaded(u);
            loaded(v);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              u[i] = __float_as_uint(fmaf(ca, __uint_as_float(u[i]), cb * __uint_as_float(v[i])));
          } else {
            tmem_wait_ld();
            loaded(u);
#pragma unroll
            for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(ca * __uint_as_float(u[i]));
          }
          if (write && sg.direct) {
            uint32_t h[16];
#pragma unroll
            for (int i = 0; i < 32; ++i) not_finite(z, __uint_as_float(u[i]));
#pragma unroll
            for (int i = 0; i < 16; ++i)
              h[i] = pack16<BF>(to_range<BF>(__uint_as_float(u[2 * i])), to_range<BF>(__uint_as_float(u[2 * i + 1])));
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(dst + c * 64 + i * 16) =
                  make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
          } else if (write) {
#pragma unroll
            for (int i = 0; i < 4; ++i) st_global_32b(dst + c * 128 + i * 32, u + 8 * i);
          }
          __syncwarp();
        }
      }
      tc_fence_before();
      mbar_arrive(bar(L::O_FREE + w));
      if (other) mbar_arrive(bar(L::O_FREE + (w ^ 1)));
      if (write) {
        if (!sg.direct)
          static_cast<float2*>(sg.ml_dst)[irow] = make_float2(M - kShift<BF>, sum);
        else if (sg.ml_dst != nullptr)
          static_cast<float*>(sg.ml_dst)[irow] = log_sum(M - kShift<BF>, sum, sees);
        report_range(z, p.err);
      }
    }
  }
}

// ---------------------------------------------------------------------------- few rows: softmax
// v[r] joined over the 32 lanes by `op`, for all r at once: halves of the rows go to halves of the
// lanes, so N values cost N - 1 exchanges (and log2(32 / N) more); lane l ends with row l % N.
template <int N, class Op>
__device__ __forceinline__ float warp_join(const float (&v)[N], int lane, Op op) {
  if constexpr (N > 1) {
    constexpr int H = N / 2;
    const bool up = (lane & H) != 0;
    float w[H];
#pragma unroll
    for (int i = 0; i < H; ++i) {
      const float send = up ? v[i] : v[i + H], keep = up ? v[i + H] : v[i];
      w[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, H));
    }
    return warp_join<H>(w, lane, op);
  } else {
    return v[0];
  }
}
// The same over the 128 threads of a warpgroup, through `ex` (a value of each warp per row).
template <int N, class Op>
__device__ __forceinline__ float group_join(const float (&v)[N], int lane, int wq, int id, float4* ex, Op op) {
  float x = warp_join<N>(v, lane, op);
#pragma unroll
  for (int d = N; d < 32; d <<= 1) x = op(x, __shfl_xor_sync(0xffffffffu, x, d));
  if (lane < N) reinterpret_cast<float*>(ex + lane)[wq] = x;
  group_sync(id);
  const float4 q = ex[lane % N];
  return op(op(q.x, q.y), op(q.z, q.w));
}

// A warpgroup's work on one segment with up to N rows (N = 4, 8, 16 or 32): thread k has key k of
// every tile and, in the end, column k of O.  False (for all threads of a warp) if a bounded wait gave up.
template <int D, bool BF, int N>
__device__ __forceinline__ bool few_segment(const PagedParams& p, const Seg& sg, uint32_t bars, uint32_t base,
                                            uint8_t* gbase, uint32_t tmem, const Waits& wctx, int w, uint32_t kv,
                                            uint32_t seg_no, uint32_t& s_no) {
  using L = Few<D>;
  constexpr uint32_t NS = L::NS;
  constexpr int KPT = L::KPT;
  auto bar = [&](int i) -> uint32_t { return bars + 8u * i; };
  const int wq = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31, key = wq * 32 + lane;
  const uint32_t lanes = (uint32_t)(wq * 32) << 16;
  const int rows = sg.rows[0];
  const int id = 1 + w;
  float4* ex = reinterpret_cast<float4*>(gbase + L::OFF_EX) + w * 64;  // [2][32]: a value of each warp per row
  uint32_t ex_no = 0;
  const auto fmax_op = [](float a, float b) { return fmaxf(a, b); };
  const auto sum_op = [](float a, float b) { return a + b; };
  // Rows are spread over registers where every key needs them (m, l) and over lanes where one value per
  // row is wanted: code that runs once per segment has to be short, it comes from far.  Rows behind
  // the last one compute along with whatever Q's buffer holds there; nothing reads them.
  // Maxima are those of the unscaled scores: a weight is 2^(scale s + shift), shift = kShift - scale max, and
  // the maximum has moved by more than kLag once s > limit = max + kLag / scale.
  const float sl2 = p.scale_log2, lag = fminf(kLag<BF> / sl2, 1e30f);
  float shift[N], limit[N], l[N];
  float m_lane = -INFINITY;  // maximum of row lane % N
#pragma unroll
  for (int r = 0; r < N; ++r) {
    shift[r] = 0.f;
    limit[r] = -INFINITY;
    l[r] = 0.f;
  }
  // A wait that gave up leaves ok false, and the segment goes on to its end all the same: the
  // barriers among the warpgroup need all of its threads.
  bool ok = true;
  const int n_tiles = sg.t1 - sg.t0;
#pragma unroll 1
  for (int t = 0; t < n_tiles; ++t, ++s_no) {
    const uint32_t n = kv + t;  // step of the phase
    const TileInfo x = tile_info<L::KT>(p, sg, sg.t0 + t);
    ok &= wait_bar(bar(L::S_FULL + 2 * w + (s_no & 1u)), s_no / 2 & 1u, wctx);
    tc_fence_after();
    float s[KPT][N];  // of keys `key` (and key + 128)
    {
      uint32_t u[KPT][N];
#pragma unroll
      for (int g = 0; g < KPT; ++g) tmem_ld<N>(tmem + lanes + L::T_S(n & 3u, g), u[g]);
      tmem_wait_ld();
#pragma unroll
      for (int g = 0; g < KPT; ++g) loaded(u[g]);
#pragma unroll
      for (int g = 0; g < KPT; ++g)
#pragma unroll
        for (int r = 0; r < N; ++r) s[g][r] = __uint_as_float(u[g][r]);
    }
    // keys that a row does not see; all rows see the same ones, except own keys with several causal tokens
    if (!x.pre && p.causal && p.T > 1) {
      const int lim0 = sg.len - p.T + 1 - x.k0;  // of the first token
      if (lim0 < L::KT) {
        int tok = 0;
#pragma unroll
        for (int r = 0; r < N; ++r) {
#pragma unroll
          for (int g = 0; g < KPT; ++g)
            if (key + 128 * g >= lim0 + tok) s[g][r] = -INFINITY;
          if (++tok == p.T) tok = 0;
        }
      }
    } else {
#pragma unroll
      for (int g = 0; g < KPT; ++g)
        if (key + 128 * g >= x.n) {
#pragma unroll
          for (int r = 0; r < N; ++r) s[g][r] = -INFINITY;
        }
    }
    float top[N];  // the larger one of the thread's keys
    bool above = false;
#pragma unroll
    for (int r = 0; r < N; ++r) {
      top[r] = KPT == 2 ? fmaxf(s[0][r], s[KPT - 1][r]) : s[0][r];
      above |= top[r] > limit[r];
    }
    if (group_any(id, above)) {
      // a maximum has moved (always on the first tile): take the tile's maxima
      const float t_max = group_join<N>(top, lane, wq, id, ex + (ex_no++ & 1u) * 32, fmax_op);
      const float m_new = fmaxf(m_lane, t_max);
      const float m_use = m_new > m_lane + lag ? m_new : m_lane;
      const float alpha = m_use == m_lane ? 1.0f : ex2_approx((m_lane - m_use) * sl2);
      m_lane = m_use;
#pragma unroll
      for (int r = 0; r < N; ++r) {
        const float x_r = __shfl_sync(0xffffffffu, m_use, r);
        limit[r] = x_r + lag;
        shift[r] = x_r == -INFINITY ? 0.f : fmaf(-x_r, sl2, kShift<BF>);
      }
      if (t > 0) {
        // O^T holds the earlier tiles once their products have completed
        ok &= wait_bar(bar(L::P_EMPTY + ((n - 1) & 1u)), (n - 1) / 2 & 1u, wctx);
        tc_fence_after();
        float a[N];
#pragma unroll
        for (int r = 0; r < N; ++r) {
          a[r] = __shfl_sync(0xffffffffu, alpha, r);
          l[r] *= a[r];
        }
#pragma unroll
        for (int h = 0; h < L::PARTS_D; ++h) {
          uint32_t u[N];
          tmem_ld<N>(tmem + lanes + L::T_O(seg_no & 1u, h), u);
          tmem_wait_ld();
          loaded(u);
#pragma unroll
          for (int r = 0; r < N; ++r) u[r] = __float_as_uint(__uint_as_float(u[r]) * a[r]);
          tmem_st<N>(tmem + lanes + L::T_O(seg_no & 1u, h), u);
        }
        tmem_wait_st();
      }
    }
    // P^T: row r of the buffer holds the weights of query row r, 64 keys to a 128-byte row of a chunk
    if (n >= 2) ok &= wait_bar(bar(L::P_EMPTY + (n & 1u)), (n / 2 - 1) & 1u, wctx);
    // (16-byte units of a row are swizzled by the row: bits 4 - 6 of the address)
    const uint32_t pb = base + L::OFF_P + (n & 1u) * L::PBUF + (key >> 6) * L::RCHUNK + (key & 63) * 2;
#pragma unroll
    for (int g = 0; g < KPT; ++g)
#pragma unroll
      for (int r = 0; r < N; ++r) {
        const float e = ex2_approx(fmaf(s[g][r], sl2, shift[r]));
        l[r] += e;
        st_shared_u16((pb ^ ((r & 7) << 4)) + r * 128 + g * 2 * L::RCHUNK, round16<BF>(e));
      }
    if (x.n < L::KT) {
      // the tile ends behind the last token: rows x.n .. of V are whatever was there before
#pragma unroll
      for (int h = 0; h < L::PARTS; ++h) {
        const uint32_t i = (2 * n + 1) * L::PARTS + h, st = i % NS;
        ok &= wait_bar(bar(L::KV_FULL + st), i / NS & 1u, wctx);
        zero_rows(gbase + st * L::SLOT, L::PCH, L::CHUNK, KPT == 2 ? min(128, max(0, x.n - 128 * h)) : x.n);
      }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    mbar_arrive(bar(L::P_FULL + (n & 1u)));
  }
  // ---- the end of the segment: row sums over the threads, then column `key` of each row
  const float total = group_join<N>(l, lane, wq, id, ex + (ex_no++ & 1u) * 32, sum_op);  // of row lane % N
  // (results are written at once where the row has own keys only)
  const bool sees = !p.causal || sg.len - p.T + lane % N % p.T >= 0;
  const float factor = sees ? __fdividef(1.0f, total) : 0.f;
  if (key < rows) {  // (warp 0)
    if (!sg.direct)
      static_cast<float2*>(sg.ml_dst)[key] = make_float2(fmaf(m_lane, sl2, -kShift<BF>), total);
    else if (sg.ml_dst != nullptr)
      static_cast<float*>(sg.ml_dst)[key] = log_sum(fmaf(m_lane, sl2, -kShift<BF>), total, sees);
  }
  ok &= wait_bar(bar(L::O_FULL + (seg_no & 1u)), seg_no / 2 & 1u, wctx);
  tc_fence_after();
  uint32_t u[L::PARTS_D][N];
#pragma unroll
  for (int h = 0; h < L::PARTS_D; ++h) tmem_ld<N>(tmem + lanes + L::T_O(seg_no & 1u, h), u[h]);
  tmem_wait_ld();
#pragma unroll
  for (int h = 0; h < L::PARTS_D; ++h) loaded(u[h]);
  tc_fence_before();
  mbar_arrive(bar(L::O_FREE + (seg_no & 1u)));
  const bool write = D >= 128 || key < D;
  if (sg.direct) {
    uint16_t* dst = reinterpret_cast<uint16_t*>(sg.o_dst) + key;
    float z = 0.f;
#pragma unroll
    for (int r = 0; r < N; ++r) {
      const float f = __shfl_sync(0xffffffffu, factor, r);
#pragma unroll
      for (int h = 0; h < L::PARTS_D; ++h)
        if (write && r < rows) {
          const float x = __uint_as_float(u[h][r]) * f;
          not_finite(z, x);
          dst[r * D + h * 128] = round16<BF>(to_range<BF>(x));
        }
    }
    report_range(z, p.err);
  } else {
    float* dst = reinterpret_cast<float*>(sg.o_dst) + key;
#pragma unroll
    for (int r = 0; r < N; ++r)
#pragma unroll
      for (int h = 0; h < L::PARTS_D; ++h)
        if (write && r < rows) dst[r * D + h * 128] = __uint_as_float(u[h][r]);
  }
  return ok;
}

// Warps 0 - 3: copies and products.
template <int D, bool BF>
__device__ __forceinline__ void few_feed(const PagedMaps& maps, const PagedParams& p, SegRing& segs, uint32_t base,
                                         uint32_t bars, uint32_t tmem, volatile uint32_t* asked_for,
                                         const Waits& wctx) {
  using L = Few<D>;
  constexpr uint32_t NS = L::NS, NQ = L::NQ;
  constexpr int PARTS = L::PARTS;
  auto bar = [&](int i) -> uint32_t { return bars + 8u * i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Seg sg;

  if (warp == 0 || warp == 2) {
    // ===================================================== page lookup and TMA: Q and K, or V
    const int v = warp >> 1;
    const CUtensorMap* map = v ? &maps.v : &maps.k;
    const int per_chunk = L::KT / p.box_rows;  // at most 32 boxes per slot or, at d = 64, pair of slots
    const int chunk = lane / per_chunk, row0 = (lane - chunk * per_chunk) * p.box_rows;
    const bool has_box = chunk < L::PCH;
    const int page_mask = (1 << p.page_shift) - 1;
    uint32_t i = v * PARTS, seg_no = 0;  // ring index of the next tile
    uint32_t issued = 0;                 // ring index behind the last slot asked for
    bool ok = true;
    for (; ok && segs.next(sg, wctx); ++seg_no) {
      TileInfo x = tile_info<L::KT>(p, sg, sg.t0);
      int page = has_box ? look_up(p, sg, x, row0) : 0;
      if (v == 0) {
        const uint32_t qb = seg_no % NQ;
        if (seg_no >= NQ && !(ok = wait_bar(bar(L::Q_EMPTY + qb), (seg_no / NQ - 1) & 1u, wctx))) break;
        const int rows = sg.own ? p.R : p.R * p.seqs;  // (a box behind the last sequence counts in full)
        if (lane == 0) mbar_arrive_expect_tx(bar(L::Q_FULL + qb), (uint32_t)rows * 128u * L::KCH);
        __syncwarp();
        if (lane < L::KCH)
          tma_load_4d(base + L::OFF_Q + (qb * L::KCH + lane) * L::RCHUNK, sg.own ? &maps.q_own : &maps.q_pre, lane * 64,
                      0, sg.hk, sg.b, bar(L::Q_FULL + qb));
      }
      for (int t = sg.t0; t < sg.t1 && ok; ++t, i += 2 * PARTS) {
        const TileInfo y = x;
        const int cur = page;
        if (t + 1 < sg.t1) {
          x = tile_info<L::KT>(p, sg, t + 1);
          if (has_box) page = look_up(p, sg, x, row0);
        }
#pragma unroll
        for (int h = 0; h < PARTS; ++h) {
          const uint32_t st = (i + h) % NS;
          if (!(ok = wait_bar(bar(L::KV_EMPTY + st), ((i + h) / NS & 1u) ^ 1u, wctx))) break;
          // slot h: columns from 128 h on (d = 256), or keys from 128 h on (d = 64)
          const int first = L::KPT == 2 ? 128 * h : 0, col = L::KPT == 2 ? 0 : h * L::PCH;
          const int rows = min(128, max(0, y.n - first));
          if (lane == 0)
            mbar_arrive_expect_tx(bar(L::KV_FULL + st),
                                  (uint32_t)((rows + p.box_rows - 1) / p.box_rows) * p.box_rows * 128u * L::PCH);
          __syncwarp();
          if (has_box && row0 >= first && row0 < first + rows)
            tma_load_4d(base + st * L::SLOT + chunk * L::CHUNK + (row0 - first) * 128, map, (col + chunk) * 64,
                        (y.k0 + row0) & page_mask, sg.hk, cur, bar(L::KV_FULL + st));
          issued = i + h + 1;
        }
      }
    }
    if (lane == 0) asked_for[v] = issued;
    // the copies of Q have landed before the phase ends (at once, unless a wait gave up)
    if (v == 0)
      for (uint32_t k = seg_no > NQ ? seg_no - NQ : 0; k < seg_no; ++k)
        drain_wait(bar(L::Q_FULL + k % NQ), k / NQ & 1u);
  } else if (warp == 1) {
    // ===================================================== products
    const uint32_t leader = elect_one();
    constexpr uint32_t idesc_s = make_idesc(128, 0, BF, false, false);  // + columns: 16 or 32
    constexpr uint32_t idesc_o = make_idesc(128, 0, BF, true, false);
    const uint64_t dK0 = make_sdesc_sw128(base, 16, 1024);
    const uint64_t dV0 = make_sdesc_sw128(base, L::CHUNK, 1024);
    const uint64_t dQ0 = make_sdesc_sw128(base + L::OFF_Q, 16, 1024);
    const uint64_t dP0 = make_sdesc_sw128(base + L::OFF_P, 16, 1024);
    bool ok = true;
    struct Step {
      bool valid, first, last;
      uint32_t seg_no, cols;
    };
    int t = 0, n_tiles = 0;
    uint32_t n_s = 0, seg_no = 0xffffffffu, cols = 0;
    // steps of each warpgroup: it waits for its own only, so they have their own barriers
    uint32_t s_no0 = 0, s_no1 = 0;
    bool more = true;
    auto issue_s = [&]() -> Step {
      Step f{};
      if (!more) return f;
      if (t == n_tiles) {
        if (!(more = segs.next(sg, wctx))) return f;
        ++seg_no;
        t = 0;
        n_tiles = sg.t1 - sg.t0;
        cols = sg.rows[0] <= 16 ? 16 : 32;
      }
      const uint32_t qb = seg_no % NQ;
      if (t == 0 && !(ok = wait_bar(bar(L::Q_FULL + qb), seg_no / NQ & 1u, wctx))) return f;
#pragma unroll
      for (int h = 0; h < PARTS; ++h) {
        const uint32_t i = 2 * n_s * PARTS + h, st = i % NS;
        if (!(ok = wait_bar(bar(L::KV_FULL + st), i / NS & 1u, wctx))) return f;
        tc_fence_after();
        const uint64_t dk = sdesc_add(dK0, st * L::SLOT);
        const uint64_t dq = sdesc_add(dQ0, (qb * L::KCH + (L::KPT == 2 ? 0 : h * L::PCH)) * L::RCHUNK);
        const uint32_t d_s = tmem + L::T_S(n_s & 3u, L::KPT == 2 ? h : 0);
#pragma unroll 1
        for (int c = 0; c < L::PCH; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ss(d_s, sdesc_add(dk, c * L::CHUNK + k * 32), sdesc_add(dq, c * L::RCHUNK + k * 32),
                   idesc_s | (cols >> 3) << 17, (L::KPT == 2 ? 0 : h) + c + k, leader);
        mma_commit(bar(L::KV_EMPTY + st), leader);
      }
      const uint32_t w = seg_no & 1u;
      mma_commit(bar(L::S_FULL + 2 * w + ((w ? s_no1++ : s_no0++) & 1u)), leader);
      if (t == n_tiles - 1) mma_commit(bar(L::Q_EMPTY + qb), leader);
      f.valid = true;
      f.first = t == 0;
      f.last = t == n_tiles - 1;
      f.seg_no = seg_no;
      f.cols = cols;
      ++t;
      ++n_s;
      return f;
    };
    Step f0 = issue_s();
    Step f1{};
    if (ok) f1 = issue_s();
    for (uint32_t n = 0; ok && f0.valid; ++n) {
      const uint32_t par = f0.seg_no & 1u;
      if (f0.first && f0.seg_no >= 2 && !(ok = wait_bar(bar(L::O_FREE + par), (f0.seg_no / 2 - 1) & 1u, wctx))) break;
      if (!(ok = wait_bar(bar(L::P_FULL + (n & 1u)), n / 2 & 1u, wctx))) break;
#pragma unroll
      for (int h = 0; h < PARTS; ++h) {
        const uint32_t i = (2 * n + 1) * PARTS + h, st = i % NS;
        if (!(ok = wait_bar(bar(L::KV_FULL + st), i / NS & 1u, wctx))) break;
        tc_fence_after();
        const uint64_t dv = sdesc_add(dV0, st * L::SLOT);
        const uint64_t dp = sdesc_add(dP0, (n & 1u) * L::PBUF + (L::KPT == 2 ? 2 * h * L::RCHUNK : 0));
        const uint32_t d_o = tmem + L::T_O(par, L::KPT == 2 ? 0 : h);
#pragma unroll 1
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ss(d_o, sdesc_add(dv, (4 * c + k) * 2048), sdesc_add(dp, c * L::RCHUNK + k * 32),
                   idesc_o | (f0.cols >> 3) << 17, (uint32_t)!f0.first + (L::KPT == 2 ? h : 0) + c + k, leader);
        mma_commit(bar(L::KV_EMPTY + st), leader);
      }
      if (!ok) break;
      mma_commit(bar(L::P_EMPTY + (n & 1u)), leader);
      if (f0.last) mma_commit(bar(L::O_FULL + par), leader);
      f0 = f1;
      f1 = issue_s();
    }
    mma_commit(bar(L::MMA_DONE), leader);
    drain_wait(bar(L::MMA_DONE), 0);
  }
}

// Warps 4 - 11: softmax, the two warpgroups take segments in turn.
template <int D, bool BF>
__device__ __forceinline__ void few_softmax(const PagedParams& p, SegRing& segs, uint32_t base, uint8_t* gbase,
                                            uint32_t bars, uint32_t tmem, const Waits& wctx) {
  Seg sg;
  const int w = (int)(threadIdx.x >> 7) - 1;
  uint32_t kv = 0, seg_no = 0, s_no = 0;
  bool ok = true;
  for (;; kv += sg.t1 - sg.t0, ++seg_no) {
    const bool more = segs.next(sg, wctx);
    if (more && (seg_no & 1u) != (uint32_t)w) continue;
    // A segment has barriers among the four warps, so they take it together or not at all: where a wait
    // gave up in one of them, this vote ends the phase for all.
    if (group_any(1 + w, !more || !ok)) break;
    const int rows = sg.rows[0];
    ok = rows <= 4    ? few_segment<D, BF, 4>(p, sg, bars, base, gbase, tmem, wctx, w, kv, seg_no, s_no)
         : rows <= 8  ? few_segment<D, BF, 8>(p, sg, bars, base, gbase, tmem, wctx, w, kv, seg_no, s_no)
         : rows <= 16 ? few_segment<D, BF, 16>(p, sg, bars, base, gbase, tmem, wctx, w, kv, seg_no, s_no)
                      : few_segment<D, BF, 32>(p, sg, bars, base, gbase, tmem, wctx, w, kv, seg_no, s_no);
  }
}

// ---------------------------------------------------------------------------- attention
template <int D, bool BF>
__global__ void __launch_bounds__(kThreads, 1)
    fa_paged_attn_sm100_kernel(const __grid_constant__ PagedMaps maps, const __grid_constant__ PagedParams p) {
  using M = Smem<D>;
  constexpr int ITEM = 128 * Dense<D>::NWG;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bars = base + M::OFF_BAR;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + M::OFF_ABORT);
  const Waits wctx{base + M::OFF_ABORT};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Start& start = *reinterpret_cast<Start*>(gbase + M::OFF_START);

  // The joining kernel may be set up as soon as multiprocessors get free; it waits for this one's end.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x < M::NBAR) {
    // arrivals: the 128 threads of a warpgroup where P, O or statistics are handed over, the reading
    // warps of a segment, else 1
    const int i = threadIdx.x, f = i - Dense<D>::NBAR;
    using A = Dense<D>;
    using F = Few<D>;
    const bool group = f < 0 ? (i >= A::P_FULL && i < A::P_FULL + 4) || (i >= A::O_FREE && i < A::O_FREE + 2) ||
                                   i == A::STAT_FULL || i == A::STAT_EMPTY
                             : (f >= F::P_FULL && f < F::P_FULL + 2) || (f >= F::O_FREE && f < F::O_FREE + 2);
    const bool in_few = f < F::NBAR;
    mbar_init(bars + 8u * i, i >= M::SEG_EMPTY ? kSegReaders : group && in_few ? 128 : 1);
    fence_barrier_init();
  }
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    start.left = 0;
  }
  if (warp == 1) {
    tmem_alloc(base + M::OFF_TMEM_SLOT, 512);
    tmem_relinquish();
  }
  // ---- this CTA's part of the own line: every thread adds up the units of its share of the
  // sequences, the block scans the sums, and the thread whose share holds the part's first unit finds it
  {
    int* scan = reinterpret_cast<int*>(gbase + M::OFF_SCAN);
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
    int mine = 0;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      mine += units_of<ITEM>(p, b);
      if (blockIdx.x == 0 && p.lens[b] > ((long long)p.max_pages << p.page_shift))
        atomicExch(p.err, kDevIndex);  // a length that the table cannot hold
    }
    int x = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    if (lane == 31) scan[warp] = x;
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += scan[w];
      total += scan[w];
    }
    before += x - mine;
    const Line line(total, p.ctas);
    const int part = p.ctas - 1 - (int)blockIdx.x;
    const int lo = part < line.parts ? line.begin(part) : 0, hi = part < line.parts ? line.begin(part + 1) : 0;
    if (hi > lo && before <= lo && lo < before + mine) {
      int skip = lo - before;
      int b = b0;
#pragma unroll 1
      for (int n; b < b1 && skip >= (n = units_of<ITEM>(p, b)); ++b) skip -= n;
      const int len = own_len(p, b);
#pragma unroll 1
      for (int rc = 0; rc < p.n_rc; ++rc) {
        const int n = item_units(own_tiles(p, len, own_visible<ITEM>(p, len, rc)));
        if (skip >= n * p.H_kv) {
          skip -= n * p.H_kv;
          continue;
        }
        start.b = b;
        start.rc = rc;
        start.hk = (int)((unsigned)skip / (unsigned)n);
        start.at = skip - start.hk * n;
        start.left = hi - lo;
        break;
      }
    }
    if (threadIdx.x == 0) start.total = total;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gbase + M::OFF_TMEM_SLOT);

  // Both lines in one phase where they take the same form, else one phase each.
  const bool pre = p.packed && p.prefix_len > 0, both = !pre || p.pre_few == p.own_few;
  uint32_t smid;
  asm volatile("mov.u32 %0, %%smid;" : "=r"(smid));
  const bool own_first = (smid >> 1 & 1u) != 0;
  const int phases = both ? 1 : 2;
  volatile uint32_t* asked_for = reinterpret_cast<volatile uint32_t*>(gbase + M::OFF_ISSUED);
  // False if a wait gave up: the CTA ends then.
  auto phase_end = [&](bool few) -> bool {
    __syncwarp();
    // The phases share the ring and tensor memory: what a thread wrote to shared memory last (the few-rows
    // form's row sums lie where the dense form at d = 128 and 256 has a ring slot) comes before the next
    // phase's copies, which a barrier alone does not order.
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (!*abort_flag) return true;
    if (threadIdx.x == 0) {
      atomicExch(p.err, kDevTimeout);
      if (few)
        drain_ring<Few<D>::NS>(bars + 8u * (M::FEW_BAR + Few<D>::KV_FULL), Few<D>::PARTS, asked_for);
      else
        drain_ring<Dense<D>::NS>(bars + 8u * (M::DENSE_BAR + Dense<D>::KV_FULL), 1, asked_for);
    }
    __syncthreads();
    return false;
  };
  Seg* ring = reinterpret_cast<Seg*>(gbase + M::OFF_SEG);
  SegRing segs{ring, bars + 8u * M::SEG_FULL, bars + 8u * M::SEG_EMPTY, 0};
  if (warp < 4) {
    regs_dec<kRegsLow>();
#pragma unroll 1
    for (int phase = 0; phase < phases; ++phase) {
      const bool do_own = both || (phase == 0) == own_first, do_pre = pre && (both || !do_own);
      const bool few = do_own ? p.own_few : p.pre_few;
      if (warp == 3)
        schedule<D>(p, start, do_pre, do_own, own_first, ring, segs.full, segs.empty, segs.no,
                    abort_flag, wctx);
      else if (few)
        few_feed<D, BF>(maps, p, segs, base, bars + 8u * M::FEW_BAR, tmem, asked_for, wctx);
      else
        dense_feed<D, BF>(maps, p, segs, base, bars + 8u * M::DENSE_BAR, tmem, asked_for, wctx);
      if (!phase_end(few)) break;
    }
  } else {
    regs_inc<kRegsHigh>();
#pragma unroll 1
    for (int phase = 0; phase < phases; ++phase) {
      const bool do_own = both || (phase == 0) == own_first;
      const bool few = do_own ? p.own_few : p.pre_few;
      if (few)
        few_softmax<D, BF>(p, segs, base, gbase, bars + 8u * M::FEW_BAR, tmem, wctx);
      else
        dense_softmax<D, BF>(p, segs, gbase, bars + 8u * M::DENSE_BAR, tmem, wctx);
      if (!phase_end(few)) break;
    }
  }
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------- joining the parts
// One warp per query row.  Parts of the own keys, then of the prefix, in the order of their lines.
template <int D, bool BF>
__global__ void __launch_bounds__(256) fa_paged_join_kernel(const PagedParams p) {
  constexpr int ITEM = 128 * Dense<D>::NWG;
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int row = (int)blockIdx.x * 8 + (int)(threadIdx.x >> 5);  // (b * H + h) * T + t, fewer than 2^30
  if (row >= p.B * p.H * p.T) return;
  const int bk = (int)((unsigned)row / (unsigned)p.R);  // b * H_kv + hk
  const int r = row - bk * p.R, b = (int)((unsigned)bk / (unsigned)p.H_kv), hk = bk - b * p.H_kv;
  const int len = own_len(p, b);
  // The parts are written.  Rows without a sequence wait too: a grid of them alone would otherwise end,
  // and the stream's next kernel begin, while the prefix items still write their parts.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (len < 0) return;
  const int rc = r / ITEM;
  const int nt = own_tiles(p, len, own_visible<ITEM>(p, len, rc));
  const bool pre = p.packed && p.prefix_len > 0;
  const int item = (b * p.n_rc + rc) * p.H_kv + hk;
  int2 own = make_int2(0, -1), pc = make_int2(0, -1);
  if (nt > 0) {
    own = p.seg[item];
    if (!parts_known(own.x, own.y, p.ctas)) return;  // after a wait that gave up, which is reported
    if (own.x == own.y && !pre) return;  // written at once
  }
  int pre_item = 0, pre_row = 0;
  if (pre) {
    const int g = b / p.group_seqs, in = b - g * p.group_seqs;
    pre_item = hk * p.n_groups + g;
    pre_row = (in / p.seqs) * 128 + (in % p.seqs) * p.R + r;
    const Line line(p.n_groups * p.H_kv * p.pre_tiles, p.ctas);
    pc.x = line.part_of(pre_item * p.pre_tiles);
    pc.y = line.part_of(pre_item * p.pre_tiles + p.pre_tiles - 1);
  }
  const int n_own = own.y - own.x + 1, n = n_own + pc.y - pc.x + 1;
  const int own_items = p.packed ? p.B * p.n_rc * p.H_kv : 0, pre_items = p.n_groups * p.H_kv;
  // where part i's row lies, counted in rows of its array
  auto at = [&](int i) -> long long {
    const bool o = i < n_own;
    const int2 c = o ? own : pc;
    const int part = c.x + (o ? i : i - n_own);
    const long long slot = c.x == c.y ? (o ? item : pre_item)
                                      : (o ? own_items : pre_items) + 2 * part + (part == c.x ? 1 : 0);
    return o ? slot * min(p.R, ITEM) + (r - rc * ITEM) : slot * p.pre_rows + pre_row;
  };
  float M = -INFINITY, L = 0.f, o[E];
#pragma unroll
  for (int i = 0; i < E; ++i) o[i] = 0.f;
  // floats per load; parts in flight (8: fewer warps fit, 4 us more at 10 parts)
  constexpr int V = E == 2 ? 2 : 4, G = 4;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int m32 = min(32, n - i0);
    float2 ml = make_float2(-INFINITY, 0.f);
    long long where = 0;
    if (lane < m32) {
      where = at(i0 + lane);
      ml = (i0 + lane < n_own ? p.own_ml : p.pre_ml)[where];
    }
    float c = 0.f;
    for (int k0 = 0; k0 < m32; k0 += G) {
      // O is on its way before the weights are known
      float v[G][E];
#pragma unroll
      for (int k = 0; k < G; ++k) {
        const long long wk = __shfl_sync(0xffffffffu, where, k0 + k);
        const float* src = (i0 + k0 + k < n_own ? p.own_o : p.pre_o) + wk * D + lane * E;
#pragma unroll
        for (int i = 0; i < E; i += V) {
          if (k0 + k >= m32) {
#pragma unroll
            for (int e = 0; e < V; ++e) v[k][i + e] = 0.f;
          } else if constexpr (V == 2) {
            const float2 x = *reinterpret_cast<const float2*>(src + i);
            v[k][i] = x.x, v[k][i + 1] = x.y;
          } else {
            const float4 x = *reinterpret_cast<const float4*>(src + i);
            v[k][i] = x.x, v[k][i + 1] = x.y, v[k][i + 2] = x.z, v[k][i + 3] = x.w;
          }
        }
      }
      if (k0 == 0) {
        float m = ml.x;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        const float mn = fmaxf(M, m);
        const float a = mn == -INFINITY ? 0.f : ex2_approx(M - mn);
        c = mn == -INFINITY ? 0.f : ex2_approx(ml.x - mn);
        float s = c * ml.y;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        L = fmaf(L, a, s);
        M = mn;
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] *= a;
      }
#pragma unroll
      for (int k = 0; k < G; ++k) {
        const float ck = __shfl_sync(0xffffffffu, c, k0 + k);
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = fmaf(ck, v[k][i], o[i]);
      }
    }
  }
  const bool sees = p.prefix_len > 0 || (p.causal ? len - p.T + r % p.T >= 0 : len > 0);
  const float inv = sees ? 1.0f / L : 0.f;
  float z = 0.f;
  uint32_t* dst = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.o) + ((size_t)row * D + lane * E) * 2);
#pragma unroll
  for (int i = 0; i < E; i += 2) {
    o[i] *= inv;
    o[i + 1] *= inv;
    not_finite(z, o[i]);
    not_finite(z, o[i + 1]);
    dst[i / 2] = pack16<BF>(to_range<BF>(o[i]), to_range<BF>(o[i + 1]));
  }
  report_range(z, p.err);
  if (lane == 0 && p.lse != nullptr) p.lse[row] = log_sum(M, L, sees);
}

template <int D, bool BF>
cudaError_t launch(const PagedMaps& maps, const PagedParams& p, cudaStream_t s) {
  constexpr int smem = Smem<D>::ALLOC;
  auto kernel = fa_paged_attn_sm100_kernel<D, BF>;
  static std::atomic<bool> ready[64];  // per device: the kernel's shared memory size is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !ready[dev].load(std::memory_order_acquire)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) ready[dev].store(true, std::memory_order_release);
  }
  kernel<<<p.ctas, kThreads, smem, s>>>(maps, p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const long long rows = (long long)p.B * p.H * p.T;
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((rows + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fa_paged_join_kernel<D, BF>, p);
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
