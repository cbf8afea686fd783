// axr_append_paged: new tokens of a ragged batch rotated, quantized with the Lloyd-Max codebook (write_vec.cuh) and
// written into paged pools through the block table; queries rotated into fp32 rows for the decode entry points.
//
// One thread block per token; every warp takes key heads, value heads and query rows in turn.  Keys and values keep
// the writer kernels' layout (d / 32 coordinates a lane, so that the Walsh-Hadamard butterfly runs in registers),
// queries 8 coordinates a lane.  The codes equal axr_write_keys' for the rotated key, bit for bit: the same
// quantize_lane on the same fp32 values.  HBM traffic bounds it on long chunks, launch latency on single tokens.
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

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Codes of one row to its place: lanes hold whole bytes of the bitstream when d / 32 codes fill them, else the row is
// packed through shared memory.
template <int D, int BITS>
__device__ __forceinline__ void store_codes(const int (&code)[D / 32], uint8_t* __restrict__ out, int lane,
                                            uint8_t* scratch) {
  constexpr int VPL = D / 32, N = VPL * BITS;
  if constexpr (N == 8 || N == 16) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) w |= static_cast<uint32_t>(code[i]) << (i * BITS);
    if constexpr (N == 8) out[lane] = static_cast<uint8_t>(w);
    else reinterpret_cast<uint16_t*>(out)[lane] = static_cast<uint16_t>(w);
  } else {
    __syncwarp();  // the previous row's bytes are read
#pragma unroll
    for (int i = 0; i < VPL; ++i) scratch[lane * VPL + i] = static_cast<uint8_t>(code[i]);
    __syncwarp();
    pack_row<D, BITS>(scratch, out, lane);
  }
}

template <typename T, int D, int BITS, bool VQ>
__global__ void __launch_bounds__(kThreads)
append_kernel(const __grid_constant__ PagedNew p, const __grid_constant__ AppendArgs a) {
  constexpr int VPL = D / 32, R = D * BITS / 8, LPR = D / 8, RPW = 32 / LPR;
  __shared__ uint8_t scratch[kWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t tok = blockIdx.x;
  int b = static_cast<int>(tok);
  if (p.cu) b = last_at_most(p.B, tok, lane, [&](int s) { return static_cast<int64_t>(p.cu[s]); });
  const NewSpan sp = new_span(p, b);
  if (tok < sp.first || tok >= sp.first + sp.count) return;  // a token past the last sequence
  const int64_t pos64 = static_cast<int64_t>(sp.pos0) + (tok - sp.first);
  if (pos64 < 0) return;
  const int64_t rpos = p.positions ? static_cast<int64_t>(p.positions[tok]) : pos64;
  int64_t row = -1;
  if (pos64 < sp.len && !(p.cos_sin && (rpos < 0 || rpos >= p.max_pos)))
    row = page_row(p, b, static_cast<int>(pos64), a.Hkv);
  if (row < 0) {
    if (threadIdx.x == 0) atomicOr(p.status, kStatusBadIndex);
    return;  // uniform over the block
  }
  row += pos64 & ((1 << p.shift) - 1);

  if (a.q) {
    Turn<8> t;
    const int e0 = 8 * (lane % LPR);
    t.load(p, rpos, e0, true);
    const T* src = static_cast<const T*>(a.q) + tok * a.q_stride + e0;
    float* dst = a.q_out + tok * a.Hq * D + e0;
    constexpr int U = 2;
    for (int h0 = warp * RPW; h0 < a.Hq; h0 += kWarps * RPW * U) {
      Raw8<T> r[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * kWarps * RPW + lane / LPR;
        if (h < a.Hq) r[u].load(src + static_cast<int64_t>(h) * D);
        else r[u].zero();
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = h0 + u * kWarps * RPW + lane / LPR;
        float x[8], o[8];
        r[u].values(x);
        r[u].from_lane(lane + t.partner).values(o);
        t.apply(x, o);
        if (h < a.Hq) store8(dst + static_cast<int64_t>(h) * D, x);
      }
    }
  }

  float sg[VPL], tau[(1 << BITS) - 1];
#pragma unroll
  for (int i = 0; i < VPL; ++i) sg[i] = sign_of(a.signs[lane * VPL + i]);
#pragma unroll
  for (int k = 0; k < (1 << BITS) - 1; ++k) tau[k] = a.cb.tau[k];
  Turn<VPL> t;
  t.load(p, rpos, lane * VPL, true);
  for (int h = warp; h < a.Hkv; h += kWarps) {
    const int64_t r = row + (static_cast<int64_t>(h) << p.shift);
    float x[VPL], y[VPL];
    load_lane<T, VPL>(static_cast<const T*>(a.k) + tok * a.k_stride + static_cast<int64_t>(h) * D, lane, x);
    load_lane<T, VPL>(static_cast<const T*>(a.v) + tok * a.v_stride + static_cast<int64_t>(h) * D, lane, y);
    float o[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) o[i] = __shfl_sync(0xffffffffu, x[i], lane + t.partner);
    t.apply(x, o);
    int code[VPL];
    const float n = quantize_lane<D, BITS>(x, sg, tau, lane, code);
    store_codes<D, BITS>(code, a.kcodes + r * R, lane, scratch[warp]);
    if (lane == 0) a.knorms[r] = __float2half_rn(n);
    if constexpr (VQ) {
      const float nv = quantize_lane<D, BITS>(y, sg, tau, lane, code);
      store_codes<D, BITS>(code, static_cast<uint8_t*>(a.vals) + r * R, lane, scratch[warp]);
      if (lane == 0) a.vnorms[r] = __float2half_rn(nv);
    } else {
      __half2 w[VPL / 2];  // fp16 inputs are stored as they are, others rounded to nearest even
#pragma unroll
      for (int i = 0; i < VPL; i += 2) w[i / 2] = __floats2half2_rn(y[i], y[i + 1]);
      __half* dst = static_cast<__half*>(a.vals) + r * D + lane * VPL;
      if constexpr (VPL == 4) *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(w);
      else *reinterpret_cast<__half2*>(dst) = w[0];
    }
  }
}

template <typename T, int D, int BITS>
axr_status launch(bool vq, const PagedNew& p, const AppendArgs& a, cudaStream_t st, const char* w) {
  const unsigned grid = static_cast<unsigned>(p.n_tok);
  if (vq) append_kernel<T, D, BITS, true><<<grid, kThreads, 0, st>>>(p, a);
  else append_kernel<T, D, BITS, false><<<grid, kThreads, 0, st>>>(p, a);
  return check_launch(w);
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
