// axr_q8_attend_paged: argument checks, the choice of kernels and the split of the token axis.
#include <algorithm>
#include <cmath>

#include "axr_host.h"
#include "paged_host.h"
#include "q8_attend.cuh"

namespace axr {
namespace {

// Kernel and workspace of a call.
struct Q8Plan {
  Q8Tiles tl;
  int nrg;        // row groups of 8 of a tile
  int grid;       // q8_decode: thread blocks
  SplitPlan sp;   // q8_prefill
  size_t parts;   // partial rows in the workspace
};

// Sequences of few query rows among longer ones (decoding sequences in a batch of prompt chunks): the warp-MMA kernel
// takes those of up to 8 rows (one token from 8 heads of a group on) and the tcgen05 kernel, which would run a 256-row
// tile for each, the others.  The host knows no lengths, so the second launch is made where the mean length is below
// half of the longest (32 / 8 heads, d = 128, bf16: 63 single tokens and a chunk of 512 on up to 4096 keys 192 -> 149 us,
// 31 and a chunk of 2048 180 -> 162 us, 32 single tokens without a bound on max_q 94 -> 52 us; four ragged chunks, none
// of them short, 168 -> 171 us).
int short_tokens(int64_t n_tok, int B, int max_q, int G) {
  if (2 * n_tok >= static_cast<int64_t>(B) * max_q) return 0;
  return G <= 8 ? 8 / G : 1;
}

// The warp-MMA kernel: one block per SM, fewer when shares of two key tiles would not fill them.
Q8Plan plan_decode(int64_t n_tok, int B, int G, int Hkv, int T, bool one, int max_q) {
  Q8Plan pl;
  pl.nrg = (one ? static_cast<int64_t>(max_q) * G <= 8 : G <= 8 && n_tok <= B) ? 1 : 2;
  pl.tl.tpt = 8 * pl.nrg / G;
  pl.tl.one = one;
  pl.tl.skip_long = false;
  pl.tl.skip_short = 0;
  pl.tl.tiles = one ? B : n_tok / pl.tl.tpt + B;
  pl.sp.splits = 1;
  pl.sp.chunk = 0;
  const int64_t shares = (pl.tl.tiles * Hkv * ((static_cast<int64_t>(T) + 31) / 32) + 1) / 2;
  pl.grid = static_cast<int>(shares < 1 ? 1 : shares < kSmCount ? shares : kSmCount);
  pl.parts = static_cast<size_t>(pl.grid) * q8_decode_warps(pl.nrg) * 2 * 8 * pl.nrg;
  return pl;
}

constexpr int64_t kMaxPartials = 16 * kSmCount * kQ8PrefillRows;  // 315 MB of workspace at d = 128

// The tcgen05 kernel: tiles of 256 rows, one thread block per SM, a tile a sequence where max_q allows it.  The split of
// the token axis minimises an estimate in units of one key tile (128 tokens, about 2 us of a full row tile):
//   waves (keys / splits + 5.5 + 5.4 fill) + 2.1   with fill the rows in use of a tile, the last two terms if split,
// fitted to 66 calls of 1 to 16 sequences and 16 to 4096 tokens each on 2048 to 32768 keys, timed at up to nine splits
// (7 % rms; the choice is 0.5 % above the best split on average, 9 % at most.  An estimate with 2 and 3 fill in their
// places split two chunks of 2048 on 8192 keys, 459 us, in two, 583 us).  The host knows no lengths: sequences are taken
// to be T long, and how many tiles have work is estimated, with every sequence, or, beside a launch for those of up to
// `few` tokens, as many longer ones as there must be.  (A count of the numbered tiles instead of those with work split 148
// units of 64 key tiles in four: 173 against 117 us.)
// Blocks without work cost about one unit a wave of SMs and split, and from 9 splits on, where the merge takes a block a
// row, a row costs 53 / 10^5, one without work half of it (59 single tokens and a chunk of 64 on 32768 keys: 8 splits
// 184 us, 10 splits 251 us; 15 single tokens: 16 splits 112 us, 8 splits 120 us).
// The workspace holds a partial for each query row and split, and a split stops at kMaxPartials of them.  (A bound on the
// numbered tiles, with work or without, left the chunk beside 199 single tokens in one piece: 751 against 415 us.)
Q8Plan plan_prefill(int64_t n_tok, int B, int G, int Hkv, int T, int max_q, int few) {
  Q8Plan pl;
  pl.nrg = kQ8PrefillRows / 8;
  pl.tl.tpt = kQ8PrefillRows / G;
  pl.tl.one = max_q <= pl.tl.tpt;
  pl.tl.skip_long = false;
  pl.tl.skip_short = few;
  pl.tl.tiles = pl.tl.one ? B : n_tok / pl.tl.tpt + B;
  const int64_t least = std::max<int64_t>(1, (n_tok - static_cast<int64_t>(few) * B + max_q - 1) / max_q);
  const int64_t seqs = few ? least : B;
  const int64_t live =
      pl.tl.one ? seqs : std::min(n_tok / pl.tl.tpt + seqs, seqs * ((max_q - 1) / pl.tl.tpt + 1));
  const int64_t units = live * Hkv, total = (static_cast<int64_t>(T) + 127) / 128, rows = n_tok * G * Hkv;
  const double fill = std::min(1.0, static_cast<double>(n_tok) * G / (static_cast<double>(live) * kQ8PrefillRows));
  const double keys = std::max(0.0, T - 0.5 * static_cast<double>(n_tok) / B) / 128;  // causal rows: half of the new ones
  const double idle = static_cast<double>(pl.tl.tiles * Hkv - units) / kSmCount;
  const double idle_rows = idle * kSmCount * std::min(max_q, pl.tl.tpt) * G;
  double best = 0;
  for (int64_t s = 1; s == 1 || (s <= total / 2 && s <= 256 && rows * s <= kMaxPartials); ++s) {
    const int64_t per = (total + s - 1) / s, splits = (total + per - 1) / per;
    const double waves = static_cast<double>((units * splits + kSmCount - 1) / kSmCount);
    double cost = waves * (std::min(static_cast<double>(per), keys / splits) + 5.5) + idle * splits;
    if (splits > 1) cost += waves * 5.4 * fill + 2.1;
    if (splits > 8) cost += 53e-5 * (rows + 0.5 * idle_rows);
    if (s == 1 || cost < best) {
      best = cost;
      pl.sp.splits = static_cast<int>(splits);
      pl.sp.chunk = static_cast<int>(per * 128);
    }
  }
  pl.grid = 0;
  pl.parts = pl.sp.splits == 1 ? 0 : static_cast<size_t>(rows) * pl.sp.splits;
  return pl;
}

size_t partial_bytes(const Q8Plan& pl, int d) {
  return (pl.parts * (static_cast<size_t>(d) + 2) * sizeof(float) + 255) / 256 * 256;
}

bool one_tile(bool ragged, int max_q, int G) { return !ragged || (max_q > 0 && static_cast<int64_t>(max_q) * G <= 16); }

}  // namespace
}  // namespace axr

extern "C" size_t axr_q8_attend_workspace_bytes(int64_t n_tok, int max_q, int B, int Hq, int Hkv, int T, int d) {
  using namespace axr;
  if (n_tok <= 0 || n_tok > 0x7fffffff || B <= 0 || Hkv <= 0 || Hq <= 0 || Hq % Hkv || Hq / Hkv > 16 || T < 0 ||
      d <= 0 || max_q < 0 || B > kMaxSeqs)
    return 0;
  if (T == 0) T = 1;
  const int G = Hq / Hkv;
  if (max_q == 0 || max_q > n_tok) max_q = static_cast<int>(n_tok);
  const bool one = one_tile(true, max_q, G);
  const size_t x = partial_bytes(plan_decode(n_tok, B, G, Hkv, T, one, max_q), d);
  if (one) return x;
  const int few = short_tokens(n_tok, B, max_q, G);
  const size_t y = partial_bytes(plan_prefill(n_tok, B, G, Hkv, T, max_q, few), d);
  const size_t z = few ? partial_bytes(plan_decode(n_tok, B, G, Hkv, T, true, few), d) : 0;
  return std::max({x, y, z});
}

extern "C" axr_status axr_q8_attend_paged(const void* q, axr_dtype x_dtype, int64_t q_stride, const uint8_t* kcodes,
                                          const float* kscales, const uint8_t* vcodes, const float* vscales,
                                          int kind, const int32_t* block_table, int max_blocks, int block_tokens,
                                          int num_blocks, const int32_t* cu_q, const int32_t* seq_lens,
                                          int64_t n_tok, int max_q, int B, int Hq, int Hkv, int T, int d, float scale,
                                          void* out, void* workspace, size_t ws_bytes, void* stream) {
  using namespace axr;
  const char* w = "axr_q8_attend_paged";
  if (x_dtype != AXR_F32 && x_dtype != AXR_F16 && x_dtype != AXR_BF16)
    return set_error(AXR_EINVAL, "%s: bad dtype", w);
  if (kind != AXR_Q8_INT && kind != AXR_Q8_E4M3) return set_error(AXR_EINVAL, "%s: bad kind %d", w, kind);
  if (n_tok < 0 || n_tok > 0x7fffffff || B < 0 || Hq <= 0 || Hkv <= 0 || Hkv > 65535 || T < 0 ||
      max_q < 0)
    return set_error(AXR_EINVAL, "%s: bad sizes n_tok=%lld max_q=%d B=%d Hq=%d Hkv=%d T=%d", w,
                     static_cast<long long>(n_tok), max_q, B, Hq, Hkv, T);
  if (B > kMaxSeqs) return set_error(AXR_EUNSUPPORTED, "%s: B=%d above %d sequences", w, B, kMaxSeqs);
  if (Hq % Hkv) return set_error(AXR_EINVAL, "%s: Hq=%d is not a multiple of Hkv=%d", w, Hq, Hkv);
  if (d != 64 && d != 128) return set_error(AXR_EUNSUPPORTED, "%s: d=%d not in {64,128}", w, d);
  const int G = Hq / Hkv;
  if (G > 16) return set_error(AXR_EUNSUPPORTED, "%s: G=%d above 16", w, G);
  if (!cu_q && n_tok != B)
    return set_error(AXR_EINVAL, "%s: without cu_q there is one token per sequence (n_tok=%lld, B=%d)", w,
                     static_cast<long long>(n_tok), B);
  int shift = 0;
  axr_status st = check_table(w, block_table, max_blocks, block_tokens, num_blocks, &shift);
  if (st != AXR_OK) return st;
  if (static_cast<int64_t>(num_blocks) * Hkv * (block_tokens / 16) > 0x7fffffff)
    return set_error(AXR_EUNSUPPORTED, "%s: the pools have more than 2^31 scale blocks", w);
  if (static_cast<int64_t>(T) > static_cast<int64_t>(max_blocks) * block_tokens)
    return set_error(AXR_EINVAL, "%s: T=%d exceeds max_blocks=%d x block_tokens=%d", w, T, max_blocks, block_tokens);
  if (!std::isfinite(scale)) return set_error(AXR_EINVAL, "%s: scale is not finite", w);
  if (n_tok == 0 || B == 0) return set_error(AXR_OK, "");
  if (!q || !kcodes || !kscales || !vcodes || !vscales || !out) return set_error(AXR_EINVAL, "%s: null pointer", w);
  if (!aligned(q, 16) || !aligned(kcodes, 16) || !aligned(vcodes, 16) || !aligned(kscales, 4) ||
      !aligned(vscales, 4) || !aligned(out, 16) || (cu_q && !aligned(cu_q, 4)) || (seq_lens && !aligned(seq_lens, 4)))
    return set_error(AXR_EINVAL, "%s: misaligned pointer", w);
  if (q_stride < static_cast<int64_t>(Hq) * d || q_stride % (16 / static_cast<int64_t>(dtype_bytes(x_dtype))))
    return set_error(AXR_EINVAL, "%s: the token stride is below a token's heads or not a multiple of 16 bytes", w);
  if (!cu_q) max_q = 1;
  if (max_q == 0 || max_q > n_tok) max_q = static_cast<int>(n_tok);
  Q8Attend a;
  memset(&a, 0, sizeof(a));
  a.q = q; a.q_stride = q_stride; a.kcodes = kcodes; a.vcodes = vcodes; a.kscales = kscales; a.vscales = vscales;
  a.table = block_table; a.cu = cu_q; a.seq_lens = seq_lens; a.out = out; a.n_tok = n_tok;
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.G = G; a.T = T; a.max_blocks = max_blocks; a.shift = shift;
  a.num_blocks = num_blocks; a.mult = scale * kQ8Log2e;
  // up to 16 query rows per sequence and KV head: the warp-MMA kernel, one tile a sequence; more: the tcgen05 kernel,
  // or, for fp32 queries and outputs (which its fp16 weights could not serve), the warp-MMA kernel over flat tiles
  const bool one = one_tile(cu_q != nullptr, max_q, G), prefill = !one && x_dtype != AXR_F32;
  const int few_tokens = prefill ? short_tokens(n_tok, B, max_q, G) : 0;
  const Q8Plan pl = prefill ? plan_prefill(n_tok, B, G, Hkv, T > 0 ? T : 1, max_q, few_tokens)
                            : plan_decode(n_tok, B, G, Hkv, T > 0 ? T : 1, one, max_q);
  Q8Plan few;  // the short sequences' plan, beside pl
  if (few_tokens) {
    few = plan_decode(n_tok, B, G, Hkv, T > 0 ? T : 1, true, few_tokens);
    few.tl.skip_long = true;
  }
  const auto too_many = [&](const Q8Plan& x) {
    return x.tl.tiles * Hkv * 8 * x.nrg > 0x7fffffff || x.tl.tiles * Hkv * x.sp.splits > 0x7fffffff;
  };
  if (too_many(pl) || (few_tokens && too_many(few))) return set_error(AXR_EUNSUPPORTED, "%s: too many rows", w);
  // the two kernels of a mixed batch run after one another and share the workspace
  const size_t need = std::max(partial_bytes(pl, d), few_tokens ? partial_bytes(few, d) : 0);
  if (need) {
    if (!workspace || ws_bytes < need)
      return set_error(AXR_EWORKSPACE, "%s: workspace of %zu bytes, need %zu", w, workspace ? ws_bytes : 0, need);
    if (!aligned(workspace, 16)) return set_error(AXR_EINVAL, "%s: workspace not 16-byte aligned", w);
  }
  a.status = status_word();
  if (!a.status) return set_error(AXR_ECUDA, "%s: the status word has no device address", w);
  const auto use = [&](const Q8Plan& x) {
    a.splits = x.sp.splits;
    a.chunk = x.sp.chunk;
    a.rows = std::min(max_q, x.tl.tpt) * G;
    a.ws_o = static_cast<float*>(workspace);
    a.ws_m = a.ws_o + x.parts * d;
    a.ws_l = a.ws_m + x.parts;
  };
  cudaStream_t s = as_stream(stream);
  if (few_tokens) {
    use(few);
    st = q8_decode_launch(x_dtype, d, kind == AXR_Q8_INT, few.nrg, few.grid, a, few.tl, s, w);
    if (st != AXR_OK) return st;
  }
  use(pl);
  if (prefill) return q8_prefill_launch(x_dtype == AXR_F16, d, kind == AXR_Q8_INT, a, pl.tl, s, w);
  return q8_decode_launch(x_dtype, d, kind == AXR_Q8_INT, pl.nrg, pl.grid, a, pl.tl, s, w);
}
