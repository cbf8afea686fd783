// New tokens of a ragged batch on their way into a paged cache: which sequence and position a token has, where its
// rows live in the pools, and the position rotation of its query and key.
//
// Sequence b's new tokens are the flat tokens cu[b] .. cu[b + 1) - 1 (token b alone without cu), the last of them at
// cache position len_b - 1.  The rotation takes coordinate pairs (j, j + rot / 2), or (2 j, 2 j + 1) when interleaved,
// j < rot / 2:
//   y_a = a c_j - b s_j,   y_b = b c_j + a s_j
// with c_j, s_j from the caller's fp32 table.  Each product and sum is rounded by itself (no fused multiply-add), so
// that the codes formed from the rotated values are reproducible from the definition with plain fp32 operations.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "axr_common.cuh"

namespace axr {

constexpr unsigned kStatusBadIndex = AXR_STATUS_BAD_INDEX;

struct PagedNew {
  const int32_t* cu;         // [B + 1] first flat token of each sequence, or null: one token per sequence
  const int32_t* seq_lens;   // [B] lengths, the new tokens included
  const int32_t* positions;  // [n_tok] rotation positions, or null: the cache positions
  const int32_t* table;      // [B, max_blocks]
  const float* cos_sin;      // [max_pos, rot]: rot / 2 cosines, then rot / 2 sines; null: no rotation
  int64_t max_pos;
  int64_t n_tok;
  int B, max_blocks, shift, num_blocks, rot, interleaved;
  unsigned int* status;
};

// The last b in [0, B) with first(b) <= key, where first is non-decreasing and first(0) <= key.  One warp: each lane
// tests one candidate a round, so B sequences take ceil(B / 32) independent loads instead of log2 B dependent ones.
template <class First>
__device__ __forceinline__ int last_at_most(int B, int64_t key, int lane, First first) {
  int n = 0;
  for (int b0 = 0; b0 < B; b0 += 32) {
    const int b = b0 + lane;
    n += __popc(__ballot_sync(0xffffffffu, b < B && first(b) <= key));
  }
  return n > 0 ? n - 1 : 0;
}

// A sequence's new tokens: flat tokens [first, first + count), cache positions [pos0, pos0 + count).
struct NewSpan {
  int64_t first;
  int count, pos0, len;
};

__device__ __forceinline__ NewSpan new_span(const PagedNew& p, int b) {
  NewSpan s;
  const int cap = p.max_blocks << p.shift;
  s.len = p.seq_lens[b];
  int64_t lo = b, hi = static_cast<int64_t>(b) + 1;
  if (p.cu) {
    lo = p.cu[b];
    hi = p.cu[b + 1];
  }
  if (lo < 0 || hi > p.n_tok || hi < lo) lo = hi = 0;  // an inconsistent table has no new tokens here
  s.first = lo;
  s.count = static_cast<int>(hi - lo);
  s.pos0 = s.len - s.count;
  if (s.len > cap) s.len = cap;  // what lies past the table's reach is skipped (and flagged by the caller)
  return s;
}

// Row of (block of position pos, KV head 0) in a pool counted in tokens, or -1 if the table holds no valid block.
__device__ __forceinline__ int64_t page_row(const PagedNew& p, int b, int pos, int Hkv) {
  const int page = p.table[static_cast<size_t>(b) * p.max_blocks + (pos >> p.shift)];
  if (page < 0 || page >= p.num_blocks) return -1;
  return (static_cast<int64_t>(page) * Hkv) << p.shift;
}

// ---- rows of 8 coordinates a lane --------------------------------------------------------------------------------

__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8], const __half*) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8], const __nv_bfloat16*) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}

// 8 coordinates as they lie in memory: one 16-byte word for 2-byte types, two for fp32
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) == 4 ? 2 : 1];
  __device__ __forceinline__ void load(const T* p) {
    w[0] = __ldg(reinterpret_cast<const uint4*>(p));
    if constexpr (sizeof(T) == 4) w[1] = __ldg(reinterpret_cast<const uint4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() {
    w[0] = make_uint4(0, 0, 0, 0);
    if constexpr (sizeof(T) == 4) w[1] = make_uint4(0, 0, 0, 0);
  }
  // the same lane-slice of the row's other half (the rotation's partner), from lane `src`
  __device__ __forceinline__ Raw8 from_lane(int src) const {
    Raw8 r;
    constexpr int N = sizeof(T) == 4 ? 2 : 1;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      r.w[i].x = __shfl_sync(0xffffffffu, w[i].x, src);
      r.w[i].y = __shfl_sync(0xffffffffu, w[i].y, src);
      r.w[i].z = __shfl_sync(0xffffffffu, w[i].z, src);
      r.w[i].w = __shfl_sync(0xffffffffu, w[i].w, src);
    }
    return r;
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    if constexpr (sizeof(T) == 4) {
      v[0] = __uint_as_float(w[0].x); v[1] = __uint_as_float(w[0].y);
      v[2] = __uint_as_float(w[0].z); v[3] = __uint_as_float(w[0].w);
      v[4] = __uint_as_float(w[1].x); v[5] = __uint_as_float(w[1].y);
      v[6] = __uint_as_float(w[1].z); v[7] = __uint_as_float(w[1].w);
    } else {
      unpack8(w[0], v, static_cast<const T*>(nullptr));
    }
  }
};

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__half* p, const float (&v)[8]) {
  uint4 w;
  uint32_t* u = &w.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint4 w;
  uint32_t* u = &w.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = w;
}

// N consecutive fp32 values (N a power of two <= 8) from an address aligned to min(16, 4 N) bytes
template <int N>
__device__ __forceinline__ void load_floats(const float* p, float (&v)[N]) {
  if constexpr (N >= 4) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 f = __ldg(reinterpret_cast<const float4*>(p + i));
      v[i] = f.x; v[i + 1] = f.y; v[i + 2] = f.z; v[i + 3] = f.w;
    }
  } else if constexpr (N == 2) {
    const float2 f = __ldg(reinterpret_cast<const float2*>(p));
    v[0] = f.x; v[1] = f.y;
  } else {
    v[0] = __ldg(p);
  }
}

// The factors of one token's rotation for the N coordinates [e0, e0 + N) that a lane holds (e0 a multiple of N, N in
// {2, 4, 8}): coordinate e0 + i turns into own * c[i] + partner * s[i], the sign of the sine included.  Coordinates
// at or past rot stay as they are (rot is a multiple of 16, so a lane's slice turns as a whole or not at all).
template <int N>
struct Turn {
  float c[N], s[N];
  int partner;  // lane offset of the partner slice (pairs half a rotation apart), 0 otherwise
  bool on, inter;
  __device__ __forceinline__ void load(const PagedNew& p, int64_t pos, int e0, bool active) {
    const int h = p.rot >> 1;
    const bool upper = e0 >= h, inside = p.cos_sin != nullptr && e0 < p.rot;
    inter = p.interleaved != 0;
    partner = inside && !inter ? (upper ? -h / N : h / N) : 0;
    on = inside && active;
    if (!on) return;
    const float* row = p.cos_sin + pos * p.rot;
    if (inter) {
      float cc[N / 2], ss[N / 2];
      load_floats(row + (e0 >> 1), cc);
      load_floats(row + h + (e0 >> 1), ss);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        c[i] = cc[i >> 1];
        s[i] = i & 1 ? ss[i >> 1] : -ss[i >> 1];
      }
    } else {
      const int j0 = upper ? e0 - h : e0;
      load_floats(row + j0, c);
      load_floats(row + h + j0, s);
#pragma unroll
      for (int i = 0; i < N; ++i) s[i] = upper ? s[i] : -s[i];
    }
  }
  // v: own coordinates; o: the partner slice's (unused when interleaved)
  __device__ __forceinline__ void apply(float (&v)[N], const float (&o)[N]) const {
    if (!on) return;
    float y[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
      y[i] = __fadd_rn(__fmul_rn(v[i], c[i]), __fmul_rn(inter ? v[i ^ 1] : o[i], s[i]));
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = y[i];
  }
};

}  // namespace axr
