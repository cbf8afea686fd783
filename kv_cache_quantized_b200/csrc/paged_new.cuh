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
  bool cut;  // the length passes the block table's reach: what lies past it is skipped
};

// The span of the last sequence b with first(cu[b], b) <= key, where first is non-decreasing in b; without cu, of
// sequence `key`.  One warp; each lane holds one sequence's entries a round, so that finding a sequence and reading its
// entries is one round trip to memory for every 32 sequences, all in flight together.
template <class First>
__device__ __forceinline__ NewSpan find_span(const PagedNew& p, int64_t key, int lane, int& b, First first) {
  const int cap = p.max_blocks << p.shift;
  NewSpan s;
  int lo = 0, hi = 0, len = 0;
  if (p.cu) {
    b = 0;
#pragma unroll 2
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int c = min(b0 + lane, p.B - 1);
      const int l = p.cu[c], h = p.cu[c + 1], n = p.seq_lens[c];
      const unsigned who = __ballot_sync(0xffffffffu, b0 + lane < p.B && first(l, c) <= key);
      if (who || b0 == 0) {
        const int src = who ? 31 - __clz(who) : 0;
        b = b0 + src;
        lo = __shfl_sync(0xffffffffu, l, src);
        hi = __shfl_sync(0xffffffffu, h, src);
        len = __shfl_sync(0xffffffffu, n, src);
      }
    }
    if (lo < 0 || hi > p.n_tok || hi < lo) lo = hi = 0;  // an inconsistent table has no new tokens here
  } else {
    b = static_cast<int>(key);
    lo = b;
    hi = b + 1;
    len = p.seq_lens[b];
  }
  if (len < 0) {
    if (hi > lo && lane == 0) atomicOr(p.status, kStatusBadIndex);
    len = 0;
  }
  s.first = lo;
  s.count = hi - lo;
  s.pos0 = len - s.count;
  s.cut = len > cap;
  s.len = s.cut ? cap : len;
  return s;
}

// Offsets that decrease or leave the batch set the status word: the last block of a call with cu looks at all of them (in
// every warp's search the comparisons took 10 % of a step of 1024 sequences).
__device__ __forceinline__ bool check_offsets(const PagedNew& p) {
  if (!p.cu || blockIdx.x != gridDim.x - 1) return false;
  bool bad = false;
  for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
    const unsigned l = static_cast<unsigned>(p.cu[b]), h = static_cast<unsigned>(p.cu[b + 1]);  // negative ones are large
    bad |= l > h || h > static_cast<unsigned>(p.n_tok);
  }
  if (bad) atomicOr(p.status, kStatusBadIndex);
  return true;
}

// Row of (block of position pos, KV head 0) in a pool counted in tokens, or -1 if the table holds no valid block.
__device__ __forceinline__ int64_t page_row(const PagedNew& p, int b, int pos, int Hkv) {
  const int page = p.table[static_cast<size_t>(b) * p.max_blocks + (pos >> p.shift)];
  if (page < 0 || page >= p.num_blocks) return -1;
  return (static_cast<int64_t>(page) * Hkv) << p.shift;
}

// Packed fp32 product, each half rounded to nearest.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long rd;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(rd)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return *reinterpret_cast<float2*>(&rd);
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

// A new token's place: its sequence's pool row (token row of its block, KV head 0) and rotation position.
struct NewPlace {
  int64_t row, rpos;
  bool ok;
};

// One warp.  Tokens without a sequence or with a negative position are not ok; tokens whose table entry, position or
// rotation position is out of range are not ok either and set the status word.
__device__ __forceinline__ NewPlace place_of(const PagedNew& p, int64_t tok, int lane, int Hkv) {
  NewPlace r{-1, 0, false};
  int b;
  const NewSpan sp = find_span(p, tok, lane, b, [](int first, int) { return static_cast<int64_t>(first); });
  const int64_t pos = static_cast<int64_t>(sp.pos0) + (tok - sp.first);
  if (tok < sp.first || tok >= sp.first + sp.count || pos < 0) return r;
  r.rpos = p.positions ? static_cast<int64_t>(p.positions[tok]) : pos;
  r.ok = pos < sp.len && !(p.cos_sin && (r.rpos < 0 || r.rpos >= p.max_pos));
  if (r.ok) {
    r.row = page_row(p, b, static_cast<int>(pos), Hkv);
    r.ok = r.row >= 0;
    r.row += pos & ((1 << p.shift) - 1);
  }
  if (!r.ok && lane == 0) atomicOr(p.status, kStatusBadIndex);
  return r;
}

// Query rows of a token rotated by one warp: slice `part` of its heads, kQuerySlice(D) of them, 8 coordinates a lane,
// U rows a lane group.  The rows are on their way before the token's place is known.
constexpr int kQueryRows = 8;
__host__ __device__ constexpr int query_slice(int D) { return kQueryRows * (256 / D); }

template <typename T, typename TO, int D>
__device__ __forceinline__ void rotate_queries(const PagedNew& p, const void* q, int64_t q_stride, void* q_out, int Hq,
                                               int Hkv, int64_t tok, int part, int lane) {
  constexpr int U = kQueryRows, LPR = D / 8, RPW = 32 / LPR;
  const int e0 = 8 * (lane % LPR), h0 = part * query_slice(D) + lane / LPR;
  const T* src = static_cast<const T*>(q) + tok * q_stride + e0;
  TO* dst = static_cast<TO*>(q_out) + tok * Hq * D + e0;
  Raw8<T> r[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (h0 + u * RPW < Hq) r[u].load(src + static_cast<int64_t>(h0 + u * RPW) * D);
    else r[u].zero();
  }
  const NewPlace at = place_of(p, tok, lane, Hkv);
  if (!at.ok) return;  // uniform over the warp
  Turn<8> t;
  t.load(p, at.rpos, e0, true);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float x[8], o[8];
    r[u].values(x);
    r[u].from_lane(lane + t.partner).values(o);
    t.apply(x, o);
    if (h0 + u * RPW < Hq) store8(dst + static_cast<int64_t>(h0 + u * RPW) * D, x);
  }
}

}  // namespace axr
