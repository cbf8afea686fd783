// axr_q8_append_paged: new tokens rotated, quantized to 8 bits and written through the block table; queries rotated.
//
// One thread block takes one 16-token scale block of a sequence and up to HPC KV heads; further blocks rotate the queries
// (rotate_queries, a warp a token and slice of heads).  Every lane holds 8 consecutive coordinates of one token row, so
// a warp load is 16 bytes a lane and a row's rotation factors are loaded once and serve all its heads.  The scale
// block's largest magnitude goes through one redux per warp and head and a shared-memory maximum; then
//   s = max(s_old, need(amax)),  code = rne(x * (1 / s)),  and, where s grew, older codes = rne(code * (s_old * (1 / s)))
// so a scale block is one work item, whatever mix of older and new tokens it holds, and no atomics on global memory
// are needed.  Issue slots (72 %) and HBM traffic together bound long calls: q, k and v are read once and q, codes and
// scales written once, 8 x 2048 fp16 tokens of 32 / 8 heads (349 MB) in 68 us, 5.1 TB/s or 0.78 of the copy rate (two
// heads a warp and four blocks an SM; four heads and two blocks: 78 us).  A step of single tokens is three round trips to
// memory (the sequence's entries; its table entry, rows and rotation; the scales): 6 us for 64 sequences.
#include "axr_host.h"
#include "paged_new.cuh"
#include "paged_host.h"
#include "q8.cuh"

namespace axr {
namespace {

struct Q8AppendArgs {
  const void *q, *k, *v;
  void* q_out;
  int64_t q_stride, k_stride, v_stride;
  uint8_t *kcodes, *vcodes;
  float *kscales, *vscales;
  int Hq, Hkv;
};

constexpr int kAppendThreads = 256;
constexpr int kHeadsPerWarp = 2;

template <int D>
struct Q8AppendPlan {
  static constexpr int LPR = D / 8;                      // lanes per token row
  static constexpr int RPW = 32 / LPR;                   // rows per warp
  static constexpr int TW = kQ8Block / RPW;              // warps that cover the 16 tokens
  static constexpr int HG = kAppendThreads / 32 / TW;    // head groups
  static constexpr int HPC = kHeadsPerWarp * HG;         // KV heads per thread block
};

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;
}

// Zero if all of x are finite, else NaN.
__device__ __forceinline__ float finite_mark(const float (&x)[8]) {
  float2 z = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 8; i += 2) z = fma2(make_float2(x[i], x[i + 1]), make_float2(0.f, 0.f), z);
  return z.x + z.y;
}

// The new rows' codes, and where the scale grew the older rows' codes, of one head at this lane's slice; finite: so are
// all of the warp's values.
template <bool I8>
__device__ __forceinline__ void q8_store(uint8_t* dst, const float (&x)[8], float sc, float s_old, bool is_new,
                                         bool is_old, bool finite) {
  const float inv = sc > 0.f ? __fdiv_rn(1.f, sc) : 0.f;
  float y[8];
  if (is_new) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 z = mul2(make_float2(x[i], x[i + 1]), make_float2(inv, inv));
      y[i] = z.x;
      y[i + 1] = z.y;
    }
    // below what magnitudes of 2^-100 need, an older scale may be too small for the new rows: x / s leaves the codes' reach,
    // or 1 / s fp32's
    if (finite && sc >= (I8 ? 6.3e-33f : 3.1e-33f)) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(q8_pack4_finite<I8>(y), q8_pack4_finite<I8>(y + 4));
      return;
    }
  } else if (is_old && sc != s_old) {
    const uint2 w = *reinterpret_cast<const uint2*>(dst);
    const float r = __fmul_rn(s_old, inv);
    q8_values4<I8>(w.x, y);
    q8_values4<I8>(w.y, y + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(y[i], r);
  } else {
    return;
  }
  *reinterpret_cast<uint2*>(dst) = make_uint2(q8_pack4<I8>(y), q8_pack4<I8>(y + 4));
}

template <typename T, int D, bool I8>
__global__ void __launch_bounds__(kAppendThreads, sizeof(T) == 4 ? 2 : 4)
q8_append_kernel(const __grid_constant__ PagedNew p, const __grid_constant__ Q8AppendArgs a, int64_t kv_blocks,
                 int kv_parts, int q_parts) {
  using P = Q8AppendPlan<D>;
  constexpr int NH = kHeadsPerWarp;
  __shared__ unsigned int amax_s[2][P::HPC];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane / P::LPR, e0 = 8 * (lane % P::LPR);

  if (check_offsets(p)) return;
  if (blockIdx.x >= kv_blocks) {
    const int64_t u = (blockIdx.x - kv_blocks) * (kAppendThreads / 32) + warp;
    if (q_parts == 0 || u >= p.n_tok * q_parts) return;
    rotate_queries<T, T, D>(p, a.q, a.q_stride, a.q_out, a.Hq, a.Hkv, u / q_parts, static_cast<int>(u % q_parts), lane);
    return;
  }
  // the item's sequence and scale block, and the block's KV heads
  const int64_t item = static_cast<int64_t>(blockIdx.x) / kv_parts;
  const int part = static_cast<int>(blockIdx.x % kv_parts);
  int b;
  auto start = [](int first, int s) { return static_cast<int64_t>(first >> 4) + 2 * s; };
  const NewSpan sp = find_span(p, item, lane, b, start);
  const int j = p.cu ? static_cast<int>(item - start(static_cast<int>(sp.first), b)) : 0;
  const int lo = max(sp.pos0, 0);
  const int64_t blk64 = static_cast<int64_t>(lo >> 4) + j;
  if (threadIdx.x == 0 && sp.cut && sp.count > 0) atomicOr(p.status, kStatusBadIndex);
  if (j < 0 || sp.count == 0 || lo >= sp.len || blk64 * kQ8Block >= sp.len) return;  // uniform over the block
  const int t_blk = static_cast<int>(blk64) * kQ8Block;
  const int64_t row0 = page_row(p, b, t_blk, a.Hkv);
  if (row0 < 0) {
    if (threadIdx.x == 0) atomicOr(p.status, kStatusBadIndex);
    return;
  }
  const int off0 = t_blk & ((1 << p.shift) - 1);

  if (threadIdx.x < 2 * P::HPC) (&amax_s[0][0])[threadIdx.x] = 0u;

  // keys and values: this lane's token, NH heads
  const int slot = (warp % P::TW) * P::RPW + sub, pos = t_blk + slot;
  bool is_new = pos >= sp.pos0 && pos < sp.len;
  const bool is_old = pos < sp.pos0, any_old = t_blk < sp.pos0;
  const int64_t tok = sp.first + (pos - sp.pos0);
  int64_t rpos = pos;
  if (is_new) {
    if (p.positions) rpos = p.positions[tok];
    if (p.cos_sin && (rpos < 0 || rpos >= p.max_pos)) {
      is_new = false;
      if (lane % P::LPR == 0) atomicOr(p.status, kStatusBadIndex);
    }
  }
  const int hl0 = (warp / P::TW) * NH;                 // first head, of the block's
  const int h0 = part * P::HPC + hl0;
  Raw8<T> kr[NH], vr[NH];
  float ks_old[NH], vs_old[NH];
#pragma unroll
  for (int i = 0; i < NH; ++i) {
    const bool ok = h0 + i < a.Hkv;
    if (ok && is_new) {
      kr[i].load(static_cast<const T*>(a.k) + tok * a.k_stride + static_cast<int64_t>(h0 + i) * D + e0);
      vr[i].load(static_cast<const T*>(a.v) + tok * a.v_stride + static_cast<int64_t>(h0 + i) * D + e0);
    } else {
      kr[i].zero();
      vr[i].zero();
    }
    ks_old[i] = vs_old[i] = 0.f;
    if (ok && any_old) {
      const int64_t s = ((row0 + (static_cast<int64_t>(h0 + i) << p.shift)) + off0) >> 4;
      ks_old[i] = a.kscales[s];
      vs_old[i] = a.vscales[s];
    }
  }
  Turn<8> turn;
  turn.load(p, rpos, e0, is_new);
  __syncthreads();  // amax_s is zero

  // the largest magnitudes; infinities, which do not count, are looked for beside them and seldom found
  float kx[NH][8], mk[NH], mv[NH], mark = 0.f;
#pragma unroll
  for (int i = 0; i < NH; ++i) {
    float o[8];
    kr[i].values(kx[i]);
    kr[i].from_lane(lane + turn.partner).values(o);
    turn.apply(kx[i], o);
    vr[i].values(o);
    mark += finite_mark(kx[i]) + finite_mark(o);
    mk[i] = mv[i] = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      mk[i] = fmaxf(mk[i], fabsf(kx[i][e]));  // a NaN is dropped
      mv[i] = fmaxf(mv[i], fabsf(o[e]));
    }
  }
  const bool finite = !__any_sync(0xffffffffu, mark != 0.f);
  if (!finite) {
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      float o[8];
      vr[i].values(o);
      mk[i] = mv[i] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        mk[i] = fmaxf(mk[i], finite_abs(kx[i][e]));
        mv[i] = fmaxf(mv[i], finite_abs(o[e]));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NH; ++i) {
    // non-negative floats order as their bit patterns
    const unsigned int um = __reduce_max_sync(0xffffffffu, __float_as_uint(mk[i]));
    const unsigned int uv = __reduce_max_sync(0xffffffffu, __float_as_uint(mv[i]));
    if (lane == 0) {
      atomicMax(&amax_s[0][hl0 + i], um);
      atomicMax(&amax_s[1][hl0 + i], uv);
    }
  }
  __syncthreads();

#pragma unroll
  for (int i = 0; i < NH; ++i) {
    if (h0 + i >= a.Hkv) break;
    const float ks = fmaxf(ks_old[i], q8_need<I8>(__uint_as_float(amax_s[0][hl0 + i])));
    const float vs = fmaxf(vs_old[i], q8_need<I8>(__uint_as_float(amax_s[1][hl0 + i])));
    const int64_t row = row0 + (static_cast<int64_t>(h0 + i) << p.shift) + off0;
    float vx[8];
    vr[i].values(vx);
    q8_store<I8>(a.kcodes + (row + slot) * D + e0, kx[i], ks, ks_old[i], is_new, is_old, finite);
    q8_store<I8>(a.vcodes + (row + slot) * D + e0, vx, vs, vs_old[i], is_new, is_old, finite);
    if (warp % P::TW == 0 && lane == 0) {
      a.kscales[row >> 4] = ks;
      a.vscales[row >> 4] = vs;
    }
  }
}

template <typename T, int D>
axr_status launch(bool i8, const PagedNew& p, const Q8AppendArgs& a, cudaStream_t st, const char* w) {
  const int64_t items = p.cu ? (p.n_tok >> 4) + 2 * static_cast<int64_t>(p.B) : p.B;
  constexpr int warps = kAppendThreads / 32;
  const int kv_parts = (a.Hkv + Q8AppendPlan<D>::HPC - 1) / Q8AppendPlan<D>::HPC;
  const int q_parts = a.q ? (a.Hq + query_slice(D) - 1) / query_slice(D) : 0;
  const int64_t kv_blocks = items * kv_parts;
  const int64_t grid = kv_blocks + (p.n_tok * q_parts + warps - 1) / warps + (p.cu ? 1 : 0);  // check_offsets
  if (grid > 0x7fffffff) return set_error(AXR_EUNSUPPORTED, "%s: too many tokens and heads for one call", w);
  const unsigned g = static_cast<unsigned>(grid);
  if (i8) q8_append_kernel<T, D, true><<<g, kAppendThreads, 0, st>>>(p, a, kv_blocks, kv_parts, q_parts);
  else q8_append_kernel<T, D, false><<<g, kAppendThreads, 0, st>>>(p, a, kv_blocks, kv_parts, q_parts);
  return check_launch(w);
}

template <typename T>
axr_status by_d(int d, bool i8, const PagedNew& p, const Q8AppendArgs& a, cudaStream_t st, const char* w) {
  return d == 64 ? launch<T, 64>(i8, p, a, st, w) : launch<T, 128>(i8, p, a, st, w);
}

}  // namespace
}  // namespace axr

extern "C" axr_status axr_q8_append_paged(const void* q, const void* k, const void* v, axr_dtype x_dtype,
                                          int64_t q_stride, int64_t k_stride, int64_t v_stride, const float* cos_sin,
                                          int64_t max_pos, int rot, int interleaved, const int32_t* positions,
                                          const int32_t* cu_new, const int32_t* seq_lens, int64_t n_tok, int B,
                                          int Hq, int Hkv, int d, int kind, uint8_t* kcodes, float* kscales,
                                          uint8_t* vcodes, float* vscales, const int32_t* block_table,
                                          int max_blocks, int block_tokens, int num_blocks, void* q_out,
                                          void* stream) {
  using namespace axr;
  const char* w = "axr_q8_append_paged";
  if (kind != AXR_Q8_INT && kind != AXR_Q8_E4M3) return set_error(AXR_EINVAL, "%s: bad kind %d", w, kind);
  PagedNew p;
  axr_status st = paged_new_args(w, q, k, v, x_dtype, q_stride, k_stride, v_stride, cos_sin, max_pos, rot,
                                 interleaved, positions, cu_new, seq_lens, n_tok, B, Hq, Hkv, d, block_table,
                                 max_blocks, block_tokens, num_blocks, q_out, &p);
  if (st != AXR_OK) return st;
  if (n_tok == 0 || B == 0) return set_error(AXR_OK, "");
  if (!kcodes || !kscales || !vcodes || !vscales) return set_error(AXR_EINVAL, "%s: null pointer", w);
  if (!aligned(kcodes, 16) || !aligned(vcodes, 16) || !aligned(kscales, 4) || !aligned(vscales, 4))
    return set_error(AXR_EINVAL, "%s: misaligned pointer", w);
  if ((st = paged_new_status(w, &p)) != AXR_OK) return st;
  Q8AppendArgs a;
  a.q = q; a.k = k; a.v = v; a.q_out = q_out;
  a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
  a.kcodes = kcodes; a.vcodes = vcodes; a.kscales = kscales; a.vscales = vscales;
  a.Hq = Hq; a.Hkv = Hkv;
  const bool i8 = kind == AXR_Q8_INT;
  cudaStream_t s = as_stream(stream);
  if (x_dtype == AXR_F16) return by_d<__half>(d, i8, p, a, s, w);
  if (x_dtype == AXR_BF16) return by_d<__nv_bfloat16>(d, i8, p, a, s, w);
  return by_d<float>(d, i8, p, a, s, w);
}
