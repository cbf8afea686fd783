// Merge of the partials of attention over the 8-bit cache: weights 2^(m_k - max m).
#pragma once

#include "q8_attend.cuh"

namespace axr {

constexpr int kMergeWarps = 4;

// Merge of the n partials part(0) .. part(n - 1) of an output row by NW warps of a block: one, or all kMergeWarps, which
// deal the partials among them and add their sums in warp order.  n = 0 gives zeros.
template <typename T, int D, int NW, class Part>
__device__ __forceinline__ void q8_merge_row(const Q8Attend& a, int n, Part part, int64_t orow) {
  constexpr int V = D / 32;
  __shared__ float max_m[kMergeWarps], sum_l[kMergeWarps], sum_o[kMergeWarps][D];
  const int lane = threadIdx.x & 31, warp = NW == 1 ? 0 : threadIdx.x >> 5;
  // each warp its partials, U at a time: all loads of a group are in flight before its maximum is known
  constexpr int U = 8;
  float M = -INFINITY, L = 0.f, acc[V];
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.f;
  for (int k0 = warp; k0 < n; k0 += U * NW) {
    float m[U], l[U], y[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * NW;
      const bool on = k < n;
      const int64_t pt = part(on ? k : k0);
      m[u] = on ? __ldcg(a.ws_m + pt) : -INFINITY;
      l[u] = on ? __ldcg(a.ws_l + pt) : 0.f;
      const float* o = a.ws_o + pt * D + V * lane;
      if constexpr (V == 4) {
        const float4 q4 = __ldcg(reinterpret_cast<const float4*>(o));
        y[u][0] = q4.x; y[u][1] = q4.y; y[u][2] = q4.z; y[u][3] = q4.w;
      } else {
        const float2 q2 = __ldcg(reinterpret_cast<const float2*>(o));
        y[u][0] = q2.x; y[u][1] = q2.y;
      }
    }
    float top = M;
#pragma unroll
    for (int u = 0; u < U; ++u) top = fmaxf(top, m[u]);   // drops a NaN, which comes back in the sums
    const float back = top == -INFINITY ? 0.f : q8_ex2(M - top);
    L *= back;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] *= back;
    M = top;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool on = k0 + u * NW < n;
      const float f = !on || M == -INFINITY ? 0.f : q8_ex2(m[u] - M);
      L = fmaf(f, l[u], L);
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] = fmaf(f, y[u][e], acc[e]);
    }
  }
  if constexpr (NW == 1) {
    T* dst = static_cast<T*>(a.out) + orow * D + V * lane;
#pragma unroll
    for (int e = 0; e < V; ++e) dst[e] = from_float<T>(L == 0.f ? 0.f : acc[e] / L);
    return;
  }
  if (lane == 0) {
    max_m[warp] = M;
    sum_l[warp] = L;
  }
#pragma unroll
  for (int e = 0; e < V; ++e) sum_o[warp][V * lane + e] = acc[e];
  __syncthreads();
  const int j = threadIdx.x;
  if (j >= D) return;
  M = max_m[0];
#pragma unroll
  for (int w = 1; w < kMergeWarps; ++w) M = fmaxf(M, max_m[w]);
  float x = 0.f;
  L = 0.f;
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) {
    const float f = max_m[w] == -INFINITY ? 0.f : q8_ex2(max_m[w] - M);
    L = fmaf(f, sum_l[w], L);
    x = fmaf(f, sum_o[w][j], x);
  }
  static_cast<T*>(a.out)[orow * D + j] = from_float<T>(L == 0.f ? 0.f : x / L);
}

// Merge of q8_prefill_kernel's split partials, the first `rows` rows of each (row tile, KV head): a block a row, or, for
// up to 8 splits, a warp `each` rows.  Launched as a programmatic dependent of it.
template <typename T, int D, int NW>
__global__ void __launch_bounds__(32 * kMergeWarps)
q8_merge_kernel(const __grid_constant__ Q8Attend a, const __grid_constant__ Q8Tiles tl, int rows, int each) {
  const int per = NW == 1 ? kMergeWarps * each : 1, groups = (rows + per - 1) / per;
  const int unit = static_cast<int>(blockIdx.x) / groups, r0 = static_cast<int>(blockIdx.x) % groups * per;
  const int tile = unit / a.Hkv, hk = unit % a.Hkv;
  // every block waits, those without a row too: this grid's end stands for the attention kernel's
  const auto wait = [] { asm volatile("griddepcontrol.wait;\n" ::: "memory"); };
  int b;
  int64_t i0;
  const Q8Span sp = q8_tile_span(a, tl, tile, threadIdx.x & 31, b, i0);
  if (!q8_tile_live(a, tl, sp, i0, threadIdx.x)) return wait();
  const int nrow = min(tl.tpt, sp.count - static_cast<int>(i0)) * a.G;
  if (nrow > rows && r0 == 0 && threadIdx.x == 0) atomicOr(a.status, kStatusBadIndex);  // more tokens than max_q
  wait();  // the partials are complete and visible after this
  const int end = min(nrow, min(rows, r0 + per));
  for (int r = r0 + (NW == 1 ? static_cast<int>(threadIdx.x) >> 5 : 0); r < end; r += kMergeWarps) {
    const int64_t orow = (sp.first + i0 + r / a.G) * a.Hq + static_cast<int64_t>(hk) * a.G + r % a.G;
    q8_merge_row<T, D, NW>(a, a.splits, [&](int k) { return orow * a.splits + k; }, orow);
  }
}

}  // namespace axr
