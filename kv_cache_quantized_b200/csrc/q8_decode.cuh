// Decode attention over the paged 8-bit cache: every warp is a worker over (row tile, KV head, split) items, a row
// tile being up to 8 NRG query rows (tokens x heads of the group) of one sequence.
//
// Both products run as mma.sync.m16n8k16 on fp16 operands: the codes enter exactly, the fp32 query and the softmax
// weights as hi and lo fp16 planes that occupy rows 0..7 and 8..15 of the same A tile, so one MMA forms both partial
// sums and carries about 22 bits of each factor.  Coordinates and tokens may be summed in any order, so each lane
// reads 16-byte runs of a code row: of the key row 8 n + g the bytes [D/4 t, D/4 t + D/4), whose word s feeds k-step
// s; of the value rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9 the bytes [D/8 g, D/8 g + D/8), byte j going to n-tile j.  No
// code passes through shared memory or a shuffle twice.
#pragma once

#include "q8_merge.cuh"
#include "warp_mma.cuh"

namespace axr {

// 8-bit codes of two rows, 4 coordinates each, as 4 half2 (row a's coordinate, row b's coordinate)
template <bool I8>
__device__ __forceinline__ void q8_pairs(uint32_t a, uint32_t b, uint32_t (&h)[4]) {
  q8_halves<I8>(__byte_perm(a, b, 0x5140), h[0], h[1]);
  q8_halves<I8>(__byte_perm(a, b, 0x7362), h[2], h[3]);
}

template <typename T, int D, bool I8, int NRG>
__global__ void __launch_bounds__(128) q8_decode_kernel(const __grid_constant__ Q8Attend a, const Q8Tiles tl) {
  constexpr int KS = D / 16;       // k-steps of the score MMA, and 32-bit words of a lane's key run
  constexpr int NO = D / 8;        // n-tiles of the output
  constexpr int VB = D / 8;        // bytes of a lane's value run
  constexpr int ROWS = 8 * NRG;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t worker = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int64_t workers = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5);
  const int64_t items = tl.tiles * a.Hkv * a.splits;

  for (int64_t item = worker; item < items; item += workers) {
    const int split = static_cast<int>(item % a.splits);
    const int hk = static_cast<int>((item / a.splits) % a.Hkv);
    const int64_t tile = item / (static_cast<int64_t>(a.splits) * a.Hkv);
    int b;
    int64_t i0;                    // first query token of the tile, in its sequence
    q8_tile(a, tl, tile, lane, b, i0);
    const Q8Span sp = q8_span(a, b);
    if (!q8_tile_live(a, tl, sp, i0, lane)) continue;
    const int nrow = min(tl.tpt, sp.count - static_cast<int>(i0)) * a.G;
    const int t_end = sp.pos0 + static_cast<int>(i0) + nrow / a.G;      // keys the tile's last token sees
    const int begin = split * a.chunk, end = min(begin + a.chunk, t_end);

    // the rows of this lane: row 8 n + g of group n, its last visible key, and its query operand
    uint32_t qf[NRG][KS][4];
    float f_row[NRG];
    int lim[NRG];                  // keys t < lim are visible
    bool live[NRG];
    int64_t orow[NRG];
#pragma unroll
    for (int n = 0; n < NRG; ++n) {
      const int r = 8 * n + g;
      live[n] = r < nrow;
      const int i = static_cast<int>(i0) + (live[n] ? r / a.G : 0), h = hk * a.G + (live[n] ? r % a.G : 0);
      lim[n] = live[n] ? min(sp.pos0 + i + 1, end) : 0;
      orow[n] = (sp.first + i) * a.Hq + h;
      const T* src = static_cast<const T*>(a.q) + (sp.first + i) * a.q_stride + static_cast<int64_t>(h) * D + (D / 4) * t;
      float x[KS][4], mx = 0.f;
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[s][e] = live[n] ? to_float<T>(src[4 * s + e]) : 0.f;
          mx = fmaxf(mx, fabsf(x[s][e]));
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // a power of two that brings the row's largest magnitude to [2^13, 2^14): both planes keep their precision
      int ex = 0;
      if (mx > 0.f && isfinite(mx)) frexpf(mx, &ex);
      ex = max(-100, min(100, ex - 14));
      const float up = ldexpf(1.f, -ex);
      f_row[n] = a.mult * ldexpf(1.f, ex);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        split_h2(x[s][0] * up, x[s][1] * up, qf[n][s][0], qf[n][s][1]);
        split_h2(x[s][2] * up, x[s][3] * up, qf[n][s][2], qf[n][s][3]);
      }
    }

    float o[NRG][NO][4];
    float m_run[NRG], l_part[NRG];
    float vref = 0.f;              // power of two the weights' value scales are relative to
#pragma unroll
    for (int n = 0; n < NRG; ++n) {
      m_run[n] = -INFINITY;
      l_part[n] = 0.f;
#pragma unroll
      for (int j = 0; j < NO; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][j][e] = 0.f;
    }

    for (int t0 = begin; t0 < end; t0 += kQ8Block) {
      const int64_t row = q8_row(a, b, hk, t0);
      const float ks = a.kscales[row >> 4], vs = a.vscales[row >> 4];
      const uint8_t* kp = a.kcodes + row * D;
      const uint8_t* vp = a.vcodes + row * D;
      uint32_t kw[2][KS], vw[4][VB / 4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int s = 0; s < KS; s += 4)
          *reinterpret_cast<uint4*>(&kw[n][s]) = *reinterpret_cast<const uint4*>(kp + (8 * n + g) * D + (D / 4) * t + 4 * s);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int tok = 2 * t + (r & 1) + 8 * (r >> 1);
        if constexpr (VB == 16) *reinterpret_cast<uint4*>(vw[r]) = *reinterpret_cast<const uint4*>(vp + tok * D + VB * g);
        else *reinterpret_cast<uint2*>(vw[r]) = *reinterpret_cast<const uint2*>(vp + tok * D + VB * g);
        if (t0 + tok >= end) {  // rows no query sees may hold anything (an e4m3 NaN): their weight is zero, so are they
#pragma unroll
          for (int s = 0; s < VB / 4; ++s) vw[r][s] = 0u;
        }
      }

      // S = Q K^T for 16 tokens; lane (g, t) holds tokens 8 n' + 2 t + {0, 1} of row g
      float sc[NRG][2][4];
#pragma unroll
      for (int n = 0; n < NRG; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[n][k][e] = 0.f;
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t b0, b1;
          q8_halves<I8>(kw[k][s], b0, b1);
#pragma unroll
          for (int n = 0; n < NRG; ++n)
            mma16816(sc[n][k], qf[n][s][0], qf[n][s][1], qf[n][s][2], qf[n][s][3], b0, b1);
        }

      if (vs > vref) {  // uniform
        const float up = __uint_as_float((__float_as_uint(vs) + 0x7fffffu) & 0x7f800000u);
        const float f = vref / up;
        vref = up;
#pragma unroll
        for (int n = 0; n < NRG; ++n)
#pragma unroll
          for (int j = 0; j < NO; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][j][e] *= f;
      }
      const float vf = vref > 0.f ? vs / vref * 16384.f : 0.f;

      uint32_t pf[NRG][4];
#pragma unroll
      for (int n = 0; n < NRG; ++n) {
        float p[4], mx = -INFINITY;
        const float f = f_row[n] * ks;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tok = t0 + 8 * (e >> 1) + 2 * t + (e & 1);
          const float v = (sc[n][e >> 1][e & 1] + sc[n][e >> 1][2 + (e & 1)]) * f;
          p[e] = tok < lim[n] ? v : -INFINITY;
          mx = fmaxf(mx, p[e]);
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float m_new = fmaxf(m_run[n], mx);
        const float m_use = m_new == -INFINITY ? 0.f : m_new;
        const float alpha = exp2f(m_run[n] - m_use);
        m_run[n] = m_new;
        float ps = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] = exp2f(p[e] - m_use);
          ps += p[e];
          p[e] *= vf;
        }
        l_part[n] = l_part[n] * alpha + ps;
        if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll
          for (int j = 0; j < NO; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][j][e] *= alpha;  // rows g and g + 8 are planes of one row
        }
        split_h2(p[0], p[1], pf[n][0], pf[n][1]);
        split_h2(p[2], p[3], pf[n][2], pf[n][3]);
      }

      // O += P V
#pragma unroll
      for (int s = 0; s < VB / 4; ++s) {
        uint32_t b0[4], b1[4];
        q8_pairs<I8>(vw[0][s], vw[1][s], b0);
        q8_pairs<I8>(vw[2][s], vw[3][s], b1);
#pragma unroll
        for (int n = 0; n < NRG; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mma16816(o[n][4 * s + e], pf[n][0], pf[n][1], pf[n][2], pf[n][3], b0[e], b1[e]);
      }
    }

    // the rows' partials, or their outputs when the axis is not split; lane (g, t) holds coordinates
    // D/4 t + j (e = 0) and D/4 t + D/8 + j (e = 1)
    const float unscale = vref * (1.f / 16384.f);
#pragma unroll
    for (int n = 0; n < NRG; ++n) {
      float l = l_part[n];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if (!live[n]) continue;
      if (a.splits == 1) {
        const float f = l > 0.f ? unscale / l : 0.f;
        T* dst = static_cast<T*>(a.out) + orow[n] * D + (D / 4) * t;
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int j = 0; j < NO; ++j)
            dst[(D / 8) * e + j] = from_float<T>(l > 0.f ? (o[n][j][e] + o[n][j][2 + e]) * f : 0.f);
      } else {
        const int64_t part = ((tile * a.Hkv + hk) * ROWS + 8 * n + g) * a.splits + split;
        float* dst = a.ws_o + part * D + (D / 4) * t;
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int j = 0; j < NO; j += 4)
            *reinterpret_cast<float4*>(dst + (D / 8) * e + j) =
                make_float4((o[n][j][e] + o[n][j][2 + e]) * unscale, (o[n][j + 1][e] + o[n][j + 1][2 + e]) * unscale,
                            (o[n][j + 2][e] + o[n][j + 2][2 + e]) * unscale,
                            (o[n][j + 3][e] + o[n][j + 3][2 + e]) * unscale);
        if (t == 0) {
          a.ws_m[part] = m_run[n];
          a.ws_l[part] = l;
        }
      }
    }
  }
}

}  // namespace axr
