// Attention of the newest tokens of every sequence over a paged key/value cache, with a prefix
// that the whole batch shares:
//   o = softmax(scale q [K_prefix; K_own]^T) [V_prefix; V_own]
//
// One block per query row; its four warps take every fourth key, each with its own running
// maximum and sum, and join them through shared memory.  All arithmetic is fp32.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged.h"
#include "sm100.cuh"

namespace fa {
namespace {

__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f32(float x, __nv_bfloat16& y) { y = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f32(float x, __half& y) { y = __float2half_rn(x); }

template <int D, class T>
__global__ void __launch_bounds__(128) fa_paged_attn_rows_kernel(const PagedParams p) {
  constexpr int E = D / 32;  // elements per lane
  __shared__ float s_o[4][D], s_m[4], s_l[4];
  const long long row = blockIdx.x;  // (b * H + h) * T + t
  const int t = (int)(row % p.T);
  const int bh = (int)(row / p.T), b = bh / p.H, hk = (bh - b * p.H) / (p.H / p.H_kv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = p.lens[b];
  if (len < 0) return;
  int own = p.causal ? len - p.T + t + 1 : len;
  own = own < 0 ? 0 : own;
  const long long room = (long long)p.max_pages << p.page_shift;
  if (own > room) {
    if (threadIdx.x == 0) atomicExch(p.err, kDevIndex);
    own = (int)room;
  }
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    q[i] = to_f32(static_cast<const T*>(p.q)[row * D + lane * E + i]);
    o[i] = 0.f;
  }
  const int total = p.prefix_len + own;
  for (int j = warp; j < total; j += 4) {
    const bool pre = j < p.prefix_len;
    const int pos = pre ? j : j - p.prefix_len;
    const int e = pos >> p.page_shift;
    const int page = pre ? p.prefix_table[e] : p.table[(long long)b * p.table_stride + e];
    if (page < 0 || page >= p.num_pages) {
      if (lane == 0) atomicExch(p.err, kDevIndex);
      continue;
    }
    const long long in = pos & ((1 << p.page_shift) - 1);
    const T* k = static_cast<const T*>(p.k) + page * p.ks[0] + hk * p.ks[1] + in * p.ks[2] + lane * E;
    const T* v = static_cast<const T*>(p.v) + page * p.vs[0] + hk * p.vs[1] + in * p.vs[2] + lane * E;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) s = fmaf(q[i], to_f32(k[i]), s);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    s *= p.scale_log2;
    const float mn = fmaxf(m, s);
    const float a = exp2f(m - mn), w = exp2f(s - mn);
    m = mn;
    l = fmaf(l, a, w);
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = fmaf(o[i], a, w * to_f32(v[i]));
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int i = 0; i < E; ++i) s_o[warp][lane * E + i] = o[i];
  __syncthreads();
  float M = -INFINITY;
  for (int w = 0; w < 4; ++w) M = fmaxf(M, s_m[w]);
  float L = 0.f, c[4];
  for (int w = 0; w < 4; ++w) {
    c[w] = M == -INFINITY ? 0.f : exp2f(s_m[w] - M);
    L += c[w] * s_l[w];
  }
  for (int i = threadIdx.x; i < D; i += 128) {
    float x = 0.f;
    for (int w = 0; w < 4; ++w) x += c[w] * s_o[w][i];
    from_f32(L > 0.f ? x / L : 0.f, static_cast<T*>(p.o)[row * D + i]);
  }
  if (threadIdx.x == 0 && p.lse != nullptr)
    p.lse[row] = L > 0.f ? (M + log2f(L)) * 0.69314718055994531f : -INFINITY;
}

template <class T>
cudaError_t launch(const PagedParams& p, int d, cudaStream_t s) {
  const unsigned rows = (unsigned)(p.B * p.H) * (unsigned)p.T;
  if (d == 64)
    fa_paged_attn_rows_kernel<64, T><<<rows, 128, 0, s>>>(p);
  else if (d == 128)
    fa_paged_attn_rows_kernel<128, T><<<rows, 128, 0, s>>>(p);
  else
    fa_paged_attn_rows_kernel<256, T><<<rows, 128, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_attn(const PagedParams& p, int d, int dtype, cudaStream_t s) {
  return dtype == FA_BF16 ? launch<__nv_bfloat16>(p, d, s) : launch<__half>(p, d, s);
}

}  // namespace fa
