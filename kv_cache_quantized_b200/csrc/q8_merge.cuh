// Merge of q8_prefill_kernel's split partials.
#pragma once

#include "q8_attend.cuh"

namespace axr {

// Merge of the split partials of each live row of each (row tile, KV head): weights 2^(m_s - max m).  One block of D
// threads a row.
template <typename T, int D>
__global__ void __launch_bounds__(D) q8_merge_kernel(const __grid_constant__ Q8Attend a, const Q8Tiles tl, int rows) {
  const int64_t row = blockIdx.x;
  const int j = threadIdx.x, r = static_cast<int>(row % rows), hk = static_cast<int>((row / rows) % a.Hkv);
  int b;
  int64_t i0;
  q8_tile(a, tl, row / rows / a.Hkv, j & 31, b, i0);
  const Q8Span sp = q8_span(a, b);
  if (!q8_tile_live(a, tl, sp, i0, 1)) return;
  if (r >= min(tl.tpt, sp.count - static_cast<int>(i0)) * a.G) return;
  const float* m = a.ws_m + row * a.splits;
  const float* l = a.ws_l + row * a.splits;
  const float* o = a.ws_o + row * a.splits * D + j;
  float M = -INFINITY;
  for (int s = 0; s < a.splits; ++s) M = fmaxf(M, m[s]);
  float L = 0.f, acc = 0.f;
  if (M != -INFINITY)
    for (int s = 0; s < a.splits; ++s) {
      const float w = exp2f(m[s] - M);
      L = fmaf(w, l[s], L);
      acc = fmaf(w, o[static_cast<size_t>(s) * D], acc);
    }
  const int64_t orow = (sp.first + i0 + r / a.G) * a.Hq + static_cast<int64_t>(hk) * a.G + r % a.G;
  static_cast<T*>(a.out)[orow * D + j] = from_float<T>(L > 0.f ? acc / L : 0.f);
}

}  // namespace axr
