// axr_append_paged: new tokens of a ragged batch rotated, quantized with the Lloyd-Max codebook (write_vec.cuh) and
// written into paged pools through the block table; queries rotated into fp32 rows for the decode entry points.
//
// Every warp works alone: on a token and KH of its key and value heads, or on a token and a slice of its query rows
// (rotate_queries).  Keys and values keep the writer kernels' layout (d / 32 coordinates a lane, so that the
// Walsh-Hadamard butterfly runs in registers), queries 8 coordinates a lane; a warp's rows are all on their way before
// its token's place in the cache is known.  The codes equal axr_write_keys' for the rotated key, bit for bit: the same
// quantize_lane on the same fp32 values.  KH = 4 keeps 2 KB a warp in flight on long calls; short calls take KH = 1, a
// head a warp (chunks of 8192 fp16 tokens into 32 / 8 heads of d = 128, b = 4, fp16 values: 56 us against 76 us with
// KH = 1; a step of 8 tokens 3.8 us).  Issue slots bound the quantized heads (about 250 instructions a vector, 64 % of
// the slots busy), HBM traffic the query and fp16 value rows (243 MB: 4.3 TB/s, 0.66 of the copy rate), launch latency
// single tokens.
#include "axr_host.h"
#include "paged_host.h"
#include "paged_new.cuh"
#include "write_vec.cuh"

namespace axr {
namespace {

struct AppendArgs {
  const void *q, *k, *v;
  float* q_out;
  int64_t q_stride, k_stride, v_stride;
  uint8_t* kcodes;
  __half* knorms;
  void* vals;      // fp16 rows, or codes
  __half* vnorms;  // quantized values
  const int8_t* signs;
  int Hq, Hkv;
  Codebook cb;
};

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

// Codes of one row to its place.  A lane holds N = BITS d / 32 consecutive bits of the row's bitstream: whole bytes are
// stored as they are; otherwise neighbouring lanes join their fields to 32-bit words.
template <int D, int BITS>
__device__ __forceinline__ void store_codes(const int (&code)[D / 32], uint8_t* __restrict__ out, int lane) {
  constexpr int VPL = D / 32, N = VPL * BITS;
  uint32_t f = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) f |= static_cast<uint32_t>(code[i]) << (i * BITS);
  if constexpr (N == 8) {
    out[lane] = static_cast<uint8_t>(f);
  } else if constexpr (N == 16) {
    reinterpret_cast<uint16_t*>(out)[lane] = static_cast<uint16_t>(f);
  } else if constexpr (N % 3 == 0) {
    // fields of neighbouring lanes joined to pieces of 24 bits, P lanes apart; word w = bits [32 w, 32 w + 32) begins in
    // piece w + w / 3 and ends in the next
    constexpr int P = 24 / N;
    static_assert((P & (P - 1)) == 0, "whole pieces from a power of two of lanes");
#pragma unroll
    for (int m = 1; m < P; m <<= 1) f |= __shfl_down_sync(0xffffffffu, f, m) << (m * N);
    const int a = lane + lane / 3, r = 8 * (lane % 3);
    const uint32_t lo = __shfl_sync(0xffffffffu, f, a * P), hi = __shfl_sync(0xffffffffu, f, a * P + P);
    if (lane < N) reinterpret_cast<uint32_t*>(out)[lane] = (lo >> r) | (hi << (24 - r));
  } else {
    constexpr int GL = 32 / N;                 // lanes of a word
    static_assert(GL * N == 32, "whole words from a power of two of lanes");
    uint32_t w = f << (lane % GL * N);
#pragma unroll
    for (int m = 1; m < GL; m <<= 1) w |= __shfl_xor_sync(0xffffffffu, w, m);
    if (lane % GL == 0) reinterpret_cast<uint32_t*>(out)[lane / GL] = w;
  }
}

// Seven blocks an SM hide more of the butterflies' latency (1400 fp32 tokens of 12 heads, d = 64, b = 3: 14.2 -> 12.9 us;
// 400 bf16 tokens of 8 heads, d = 128: 7.2 -> 6.1 us); long calls with quantized values of d = 128 want the registers of
// six (4000 tokens of 8 heads: 36.0 against 36.7 us).
// Units of work: kv_units of (token, KH KV heads), then (token, slice of query heads).
template <typename T, int D, int BITS, bool VQ, int KH>
__global__ void __launch_bounds__(kThreads, KH == 4 && VQ && D == 128 ? 6 : 7)
append_kernel(const __grid_constant__ PagedNew p, const __grid_constant__ AppendArgs a, int64_t kv_units, int kv_parts,
              int q_parts) {
  constexpr int VPL = D / 32, R = D * BITS / 8;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (check_offsets(p)) return;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  if (unit >= kv_units) {
    const int64_t u = unit - kv_units;
    if (q_parts == 0 || u >= p.n_tok * q_parts) return;
    rotate_queries<T, float, D>(p, a.q, a.q_stride, a.q_out, a.Hq, a.Hkv, u / q_parts, static_cast<int>(u % q_parts),
                                lane);
    return;
  }
  const int64_t tok = unit / kv_parts;
  const int h0 = static_cast<int>(unit % kv_parts) * KH;
  const T* ks = static_cast<const T*>(a.k) + tok * a.k_stride + static_cast<int64_t>(h0) * D;
  const T* vs = static_cast<const T*>(a.v) + tok * a.v_stride + static_cast<int64_t>(h0) * D;
  float x[KH][VPL], y[KH][VPL];
#pragma unroll
  for (int i = 0; i < KH; ++i) {
    const bool on = h0 + i < a.Hkv;
    load_lane<T, VPL>(ks + (on ? i * D : 0), lane, x[i]);
    load_lane<T, VPL>(vs + (on ? i * D : 0), lane, y[i]);
  }
  float sg[VPL], tau[(1 << BITS) - 1];
#pragma unroll
  for (int i = 0; i < VPL; ++i) sg[i] = sign_of(a.signs[lane * VPL + i]);
#pragma unroll
  for (int k = 0; k < (1 << BITS) - 1; ++k) tau[k] = a.cb.tau[k];
  const NewPlace at = place_of(p, tok, lane, a.Hkv);
  if (!at.ok) return;  // uniform over the warp
  Turn<VPL> t;
  t.load(p, at.rpos, lane * VPL, true);
#pragma unroll
  for (int j = 0; j < KH; ++j) {
    if (h0 + j >= a.Hkv) break;
    const int64_t r = at.row + (static_cast<int64_t>(h0 + j) << p.shift);
    float o[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) o[i] = __shfl_sync(0xffffffffu, x[j][i], lane + t.partner);
    t.apply(x[j], o);
    int code[VPL];
    const float n = quantize_lane<D, BITS>(x[j], sg, tau, lane, code);
    store_codes<D, BITS>(code, a.kcodes + r * R, lane);
    if (lane == 0) a.knorms[r] = __float2half_rn(n);
    if constexpr (VQ) {
      const float nv = quantize_lane<D, BITS>(y[j], sg, tau, lane, code);
      store_codes<D, BITS>(code, static_cast<uint8_t*>(a.vals) + r * R, lane);
      if (lane == 0) a.vnorms[r] = __float2half_rn(nv);
    } else {
      __half2 w[VPL / 2];  // fp16 inputs are stored as they are, others rounded to nearest even
#pragma unroll
      for (int i = 0; i < VPL; i += 2) w[i / 2] = __floats2half2_rn(y[j][i], y[j][i + 1]);
      __half* dst = static_cast<__half*>(a.vals) + r * D + lane * VPL;
      if constexpr (VPL == 4) *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(w);
      else *reinterpret_cast<__half2*>(dst) = w[0];
    }
  }
}

template <typename T, int D, int BITS, bool VQ, int KH>
axr_status launch_kh(const PagedNew& p, const AppendArgs& a, cudaStream_t st, const char* w) {
  const int kv_parts = (a.Hkv + KH - 1) / KH, q_parts = a.q ? (a.Hq + query_slice(D) - 1) / query_slice(D) : 0;
  const int64_t kv_units = p.n_tok * kv_parts, units = kv_units + p.n_tok * q_parts;
  const int64_t grid = (units + kWarps - 1) / kWarps + (p.cu ? 1 : 0);  // check_offsets
  if (grid > 0x7fffffff) return set_error(AXR_EUNSUPPORTED, "%s: too many tokens and heads for one call", w);
  append_kernel<T, D, BITS, VQ, KH>
      <<<static_cast<unsigned>(grid), kThreads, 0, st>>>(p, a, kv_units, kv_parts, q_parts);
  return check_launch(w);
}

template <typename T, int D, int BITS>
axr_status launch(bool vq, const PagedNew& p, const AppendArgs& a, cudaStream_t st, const char* w) {
  // a head a warp until the warps fill the SMs twice over (about 24 resident a SM): 7104 rows.  A head / four heads a warp
  // at half, once and twice as many: b = 4 quantized values 6.0 / 7.9, 10.5 / 10.4, 20.8 / 16.7 us; fp16 values 5.8 / 6.3,
  // 9.6 / 8.1, 18.5 / 14.4 us; d = 64, b = 3 5.0 / 6.7, 9.1 / 7.6, 14.5 / 10.0 us
  const bool wide = p.n_tok * a.Hkv > static_cast<int64_t>(kSmCount) * 48;
  if (vq) return wide ? launch_kh<T, D, BITS, true, 4>(p, a, st, w) : launch_kh<T, D, BITS, true, 1>(p, a, st, w);
  return wide ? launch_kh<T, D, BITS, false, 4>(p, a, st, w) : launch_kh<T, D, BITS, false, 1>(p, a, st, w);
}

template <typename T, int D>
axr_status by_bits(int bits, bool vq, const PagedNew& p, const AppendArgs& a, cudaStream_t st, const char* w) {
  switch (bits) {
    case 1: return launch<T, D, 1>(vq, p, a, st, w);
    case 2: return launch<T, D, 2>(vq, p, a, st, w);
    case 3: return launch<T, D, 3>(vq, p, a, st, w);
    default: return launch<T, D, 4>(vq, p, a, st, w);
  }
}

template <typename T>
axr_status by_d(int d, int bits, bool vq, const PagedNew& p, const AppendArgs& a, cudaStream_t st, const char* w) {
  return d == 64 ? by_bits<T, 64>(bits, vq, p, a, st, w) : by_bits<T, 128>(bits, vq, p, a, st, w);
}

}  // namespace
}  // namespace axr

extern "C" axr_status axr_append_paged(const void* q, const void* k, const void* v, axr_dtype x_dtype,
                                       int64_t q_stride, int64_t k_stride, int64_t v_stride, const float* cos_sin,
                                       int64_t max_pos, int rot, int interleaved, const int32_t* positions,
                                       const int32_t* cu_new, const int32_t* seq_lens, int64_t n_tok, int B, int Hq,
                                       int Hkv, int d, int bits, const int8_t* signs, uint8_t* kcodes,
                                       uint16_t* knorms, axr_vkind vkind, void* values, uint16_t* vnorms,
                                       const int32_t* block_table, int max_blocks, int block_tokens, int num_blocks,
                                       float* q_out, void* stream) {
  using namespace axr;
  const char* w = "axr_append_paged";
  if (bits < 1 || bits > 4) return set_error(AXR_EUNSUPPORTED, "%s: bits=%d outside 1..4", w, bits);
  if (vkind != AXR_V_F16 && vkind != AXR_V_QUANT)
    return set_error(AXR_EINVAL, "%s: paged pools take the row value layouts", w);
  PagedNew p;
  axr_status st = paged_new_args(w, q, k, v, x_dtype, q_stride, k_stride, v_stride, cos_sin, max_pos, rot,
                                 interleaved, positions, cu_new, seq_lens, n_tok, B, Hq, Hkv, d, block_table,
                                 max_blocks, block_tokens, num_blocks, q_out, &p);
  if (st != AXR_OK) return st;
  if (n_tok == 0 || B == 0) return set_error(AXR_OK, "");
  if (!kcodes || !knorms || !signs || !values || (vkind == AXR_V_QUANT && !vnorms))
    return set_error(AXR_EINVAL, "%s: null pointer", w);
  if (!aligned(kcodes, 16) || !aligned(values, 16) || !aligned(knorms, 4) || (vnorms && !aligned(vnorms, 4)))
    return set_error(AXR_EINVAL, "%s: misaligned pointer", w);
  const Codebook* cb = codebook_for(d, bits);
  if (!cb) return set_error(AXR_EINVAL, "%s: codebook unavailable", w);
  if ((st = paged_new_status(w, &p)) != AXR_OK) return st;
  AppendArgs a;
  a.q = q; a.k = k; a.v = v; a.q_out = q_out;
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.kcodes = kcodes; a.knorms = reinterpret_cast<__half*>(knorms);
  a.vals = values; a.vnorms = reinterpret_cast<__half*>(vnorms);
  a.signs = signs; a.Hq = Hq; a.Hkv = Hkv; a.cb = *cb;
  const bool vq = vkind == AXR_V_QUANT;
  cudaStream_t s = as_stream(stream);
  if (x_dtype == AXR_F16) return by_d<__half>(d, bits, vq, p, a, s, w);
  if (x_dtype == AXR_BF16) return by_d<__nv_bfloat16>(d, bits, vq, p, a, s, w);
  return by_d<float>(d, bits, vq, p, a, s, w);
}
