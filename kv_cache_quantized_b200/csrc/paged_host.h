// Argument checks shared by the entry points that write new tokens into paged pools.
#pragma once

#include "axr_host.h"
#include "paged_new.cuh"

namespace axr {

// log2 of a valid pool block size (a power of two in [16, 2^20]), or -1.
inline int block_shift_of(int block_tokens) {
  int shift = 4;
  while (shift < 20 && (1 << shift) < block_tokens) ++shift;
  return (1 << shift) == block_tokens ? shift : -1;
}

inline axr_status check_table(const char* w, const int32_t* table, int max_blocks, int block_tokens, int num_blocks,
                              int* shift) {
  *shift = block_shift_of(block_tokens);
  if (*shift < 0)
    return set_error(AXR_EINVAL, "%s: block_tokens=%d is not a power of two in [16, 2^20]", w, block_tokens);
  if (max_blocks <= 0 || num_blocks <= 0)
    return set_error(AXR_EINVAL, "%s: bad sizes max_blocks=%d num_blocks=%d", w, max_blocks, num_blocks);
  if (static_cast<int64_t>(max_blocks) * block_tokens > (1 << 30))  // token positions are 32-bit in the kernels
    return set_error(AXR_EINVAL, "%s: max_blocks=%d x block_tokens=%d exceeds 2^30 tokens", w, max_blocks, block_tokens);
  if (!table) return set_error(AXR_EINVAL, "%s: null block table", w);
  if (!aligned(table, 4)) return set_error(AXR_EINVAL, "%s: misaligned block table", w);
  return AXR_OK;
}

// Every warp scans the batch's entries, 32 a round trip, so that a call's time has a part that grows as B^2: decode of 256
// sequences of 1000 tokens (32 / 8 heads) takes 164 us, of 1024 1.0 ms, where the attention kernel alone takes 102 and
// 388 us.
constexpr int kMaxSeqs = 1 << 14;

inline size_t dtype_bytes(axr_dtype t) { return t == AXR_F32 ? 4 : 2; }

// Everything but the pools.  Fills p (its status word through paged_new_status, the only CUDA call).
inline axr_status paged_new_args(const char* w, const void* q, const void* k, const void* v, axr_dtype x_dtype,
                                 int64_t q_stride, int64_t k_stride, int64_t v_stride, const float* cos_sin,
                                 int64_t max_pos, int rot, int interleaved, const int32_t* positions,
                                 const int32_t* cu_new, const int32_t* seq_lens, int64_t n_tok, int B, int Hq,
                                 int Hkv, int d, const int32_t* block_table, int max_blocks, int block_tokens,
                                 int num_blocks, const void* q_out, PagedNew* p) {
  if (x_dtype != AXR_F32 && x_dtype != AXR_F16 && x_dtype != AXR_BF16)
    return set_error(AXR_EINVAL, "%s: bad dtype", w);
  if (n_tok < 0 || n_tok > 0x7fffffff || B < 0 || Hkv <= 0 || Hkv > 65535)
    return set_error(AXR_EINVAL, "%s: bad sizes n_tok=%lld B=%d Hkv=%d", w, static_cast<long long>(n_tok), B, Hkv);
  if (B > kMaxSeqs) return set_error(AXR_EUNSUPPORTED, "%s: B=%d above %d sequences", w, B, kMaxSeqs);
  if (d != 64 && d != 128) return set_error(AXR_EUNSUPPORTED, "%s: d=%d not in {64,128}", w, d);
  if ((q == nullptr) != (q_out == nullptr)) return set_error(AXR_EINVAL, "%s: q and q_out go together", w);
  if (q && (Hq <= 0 || Hq % Hkv))
    return set_error(AXR_EINVAL, "%s: Hq=%d is not a positive multiple of Hkv=%d", w, Hq, Hkv);
  if (cos_sin && (rot <= 0 || rot > d || rot % 16))
    return set_error(AXR_EUNSUPPORTED, "%s: rot=%d is not a multiple of 16 in [16, d]", w, rot);
  if (cos_sin && max_pos <= 0) return set_error(AXR_EINVAL, "%s: max_pos=%lld", w, static_cast<long long>(max_pos));
  if (q && !cos_sin) return set_error(AXR_EINVAL, "%s: q without a rotation table", w);
  if (!cu_new && n_tok != B)
    return set_error(AXR_EINVAL, "%s: without cu_new there is one token per sequence (n_tok=%lld, B=%d)", w,
                     static_cast<long long>(n_tok), B);
  int shift = 0;
  const axr_status st = check_table(w, block_table, max_blocks, block_tokens, num_blocks, &shift);
  if (st != AXR_OK) return st;
  if (n_tok > 0 && B > 0) {
    if (!k || !v || !seq_lens) return set_error(AXR_EINVAL, "%s: null pointer", w);
    const int64_t vec = 16 / static_cast<int64_t>(dtype_bytes(x_dtype));
    if (!aligned(k, 16) || !aligned(v, 16) || (q && (!aligned(q, 16) || !aligned(q_out, 16))) ||
        (cos_sin && !aligned(cos_sin, 16)) || !aligned(seq_lens, 4) || (cu_new && !aligned(cu_new, 4)) ||
        (positions && !aligned(positions, 4)))
      return set_error(AXR_EINVAL, "%s: misaligned pointer", w);
    if (k_stride < static_cast<int64_t>(Hkv) * d || v_stride < static_cast<int64_t>(Hkv) * d ||
        (q && q_stride < static_cast<int64_t>(Hq) * d) || k_stride % vec || v_stride % vec || (q && q_stride % vec))
      return set_error(AXR_EINVAL, "%s: a token stride is below a token's heads or not a multiple of 16 bytes", w);
  }
  p->cu = cu_new; p->seq_lens = seq_lens; p->positions = positions; p->table = block_table; p->cos_sin = cos_sin;
  p->max_pos = max_pos; p->n_tok = n_tok; p->B = B; p->max_blocks = max_blocks; p->shift = shift;
  p->num_blocks = num_blocks; p->rot = cos_sin ? rot : 0; p->interleaved = interleaved ? 1 : 0; p->status = nullptr;
  return AXR_OK;
}

inline axr_status paged_new_status(const char* w, PagedNew* p) {
  p->status = status_word();
  return p->status ? AXR_OK : set_error(AXR_ECUDA, "%s: the status word has no device address", w);
}

}  // namespace axr
