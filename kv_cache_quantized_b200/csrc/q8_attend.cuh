// Attention over the paged 8-bit cache (q8.cuh): arguments and helpers shared by its kernels.
//
// Query row r = (token i, head g) of a sequence and KV head sees keys 0 .. pos0 + i below T, pos0 = len - count:
//   s_t = scale * ks_t (q . code^K_t),   o = sum_t 2^(s_t log2 e - m) vs_t code^V_t / sum_t 2^(s_t log2 e - m)
// with ks_t, vs_t the scales of token t's 16-token block.
#pragma once

#include "paged_new.cuh"
#include "q8.cuh"

namespace axr {

constexpr float kQ8Log2e = 1.4426950408889634f;

struct Q8Attend {
  const void* q;            // token rows of q_stride elements, [Hq, D] each
  int64_t q_stride;
  const uint8_t *kcodes, *vcodes;
  const float *kscales, *vscales;
  const int32_t* table;     // [B, max_blocks]
  const int32_t* cu;        // [B + 1] or null: one query token per sequence
  const int32_t* seq_lens;  // [B] or null: T
  void* out;                // [n_tok, Hq, D]
  float *ws_o, *ws_m, *ws_l;  // partials: [parts, D], [parts] x 2; parts as the kernel lays them out
  int64_t n_tok;
  int B, Hq, Hkv, G, T, max_blocks, shift, num_blocks;
  int splits, chunk;        // q8_prefill: the token axis as splits chunks of `chunk` tokens
  int rows;                 // q8_prefill: rows that a tile has at most, by the caller's bound on the query tokens
  float mult;               // scale * log2 e
  unsigned int* status;
};

// One sequence's query tokens and length.  Positions come from the length as it is, the keys seen from that cut to T: a
// length past T moves no token's causal limit.
struct Q8Span {
  int64_t first;    // first flat token
  int count, pos0;  // new tokens, position of the first
  __device__ __forceinline__ int keys(int T) const { return min(pos0 + count, T); }
};

// From the entries cu[b], cu[b + 1] and the length.  A sequence whose entries make no sense counts as empty; such entries,
// or a length out of range, set the status word (FLAG).
template <bool FLAG = true>
__device__ __forceinline__ Q8Span q8_span_of(const Q8Attend& a, int64_t lo, int64_t hi, int len) {
  Q8Span s;
  bool bad = false;
  if (lo < 0 || hi > a.n_tok || hi < lo) {
    lo = hi = 0;
    bad = true;
  }
  s.first = lo;
  s.count = static_cast<int>(hi - lo);
  s.pos0 = max(len, 0) - s.count;
  if (FLAG && (bad || (s.count > 0 && (len < 0 || len > a.T)))) atomicOr(a.status, kStatusBadIndex);
  return s;
}

template <bool FLAG = true>
__device__ __forceinline__ Q8Span q8_span(const Q8Attend& a, int b) {
  const int len = a.seq_lens ? a.seq_lens[b] : a.T;
  return a.cu ? q8_span_of<FLAG>(a, a.cu[b], a.cu[b + 1], len)
              : q8_span_of<FLAG>(a, b, static_cast<int64_t>(b) + 1, len);
}

// How a kernel cuts the query tokens into row tiles of up to tpt tokens (times the heads of a group).
//  one  = true:  tile b is sequence b, which has at most tpt tokens; longer sequences are another kernel's (skip_long)
//                or break the caller's bound (flagged in the status word);
//  one  = false: sequence b owns the tiles from cu[b] / tpt + b on: at most n_tok / tpt + B tiles in all, found
//                without knowing the lengths on the host.  Sequences of at most skip_short tokens are skipped (another
//                kernel's).
struct Q8Tiles {
  int64_t tiles;
  int tpt;
  bool one, skip_long;
  int skip_short;
};

// q8_decode.cu: tiles of up to 8 nrg query rows, one share of the key tiles a warp; any dtype.  The workspace holds two
// partials of 8 nrg rows for each worker.
constexpr int q8_decode_warps(int nrg) { return nrg == 1 ? 12 : 8; }  // a block
axr_status q8_decode_launch(axr_dtype dtype, int d, bool i8, int nrg, int grid, const Q8Attend& a, const Q8Tiles& tl,
                            cudaStream_t st, const char* w);

// q8_prefill.cu: tiles of up to 256 query rows on the tcgen05 tensor cores, queries and outputs fp16 (half) or bf16.
constexpr int kQ8PrefillRows = 256;
axr_status q8_prefill_launch(bool half, int d, bool i8, const Q8Attend& a, const Q8Tiles& tl, cudaStream_t st,
                             const char* w);

// Sequence and first token of a tile.  One warp.
__device__ __forceinline__ void q8_tile(const Q8Attend& a, const Q8Tiles& tl, int64_t tile, int lane, int& b,
                                        int64_t& i0) {
  b = static_cast<int>(tile);
  i0 = 0;
  if (!tl.one) {
    auto start = [&](int s) { return static_cast<int64_t>(a.cu[s]) / tl.tpt + s; };
    b = last_at_most(a.B, tile, lane, start);
    i0 = (tile - start(b)) * tl.tpt;
  }
}

// The same, and the sequence's entries, in one round trip to memory for every 32 sequences.
__device__ __forceinline__ Q8Span q8_tile_span(const Q8Attend& a, const Q8Tiles& tl, int64_t tile, int lane, int& b,
                                               int64_t& i0) {
  if (tl.one) {
    b = static_cast<int>(tile);
    i0 = 0;
    return q8_span(a, b);
  }
  const unsigned n_tok = static_cast<unsigned>(a.n_tok);
  int lo = 0, hi = 0, len = 0;
  bool bad = false;
  b = 0;
  i0 = -1;
#pragma unroll 2
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int c = min(b0 + lane, a.B - 1);
    const int l = a.cu[c], h = a.cu[c + 1], n = a.seq_lens ? a.seq_lens[c] : a.T;
    // every sequence's offsets (as unsigned, negative ones are large); lengths where a tile has them
    bad |= static_cast<unsigned>(l) > static_cast<unsigned>(h) || static_cast<unsigned>(h) > n_tok;
    const int64_t first = static_cast<int64_t>(l / tl.tpt) + c;
    const unsigned who = __ballot_sync(0xffffffffu, b0 + lane < a.B && first <= tile);
    if (who) {
      const int src = 31 - __clz(who);
      b = b0 + src;
      i0 = (tile - __shfl_sync(0xffffffffu, first, src)) * tl.tpt;
      lo = __shfl_sync(0xffffffffu, l, src);
      hi = __shfl_sync(0xffffffffu, h, src);
      len = __shfl_sync(0xffffffffu, n, src);
    }
  }
  if (bad) atomicOr(a.status, kStatusBadIndex);
  return q8_span_of(a, lo, hi, len);
}

__device__ __forceinline__ bool q8_tile_live(const Q8Attend& a, const Q8Tiles& tl, const Q8Span& sp, int64_t i0,
                                             int lane) {
  if (tl.one && sp.count > tl.tpt) {
    if (!tl.skip_long && lane == 0) atomicOr(a.status, kStatusBadIndex);
    return false;
  }
  return i0 >= 0 && i0 < sp.count && sp.count > tl.skip_short;
}

// Pool row (in tokens, KV head hk) of cache position t of sequence b; an entry outside the pools reads block 0 and
// sets the status word.
__device__ __forceinline__ int64_t q8_row(const Q8Attend& a, int b, int hk, int t) {
  int page = __ldg(a.table + static_cast<size_t>(b) * a.max_blocks + (t >> a.shift));
  if (page < 0 || page >= a.num_blocks) {
    atomicOr(a.status, kStatusBadIndex);
    page = 0;
  }
  return ((static_cast<int64_t>(page) * a.Hkv + hk) << a.shift) + (t & ((1 << a.shift) - 1));
}

__device__ __forceinline__ float q8_ex2(float x) {  // relative error 2^-22, as the planes of the queries and weights
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

}  // namespace axr
