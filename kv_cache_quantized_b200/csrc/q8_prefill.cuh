// Attention of many query tokens over the paged 8-bit cache on the tcgen05 tensor cores.
//
// One thread block takes up to 256 query rows (tokens x heads of one KV head's group) as two row tiles of 128, and a
// range of the token axis in steps of 64 keys:
//   S = Q K^T     M = 128 rows, N = 64 tokens: Q and the key codes in shared memory (fp16, K-major, 128-byte swizzle),
//                 S in tensor memory, fp32, two buffers a row tile;
//   P = 2^(ks f S - m), times vs / vref, rounded to fp16 and stored over S in tensor memory;
//   O += P V      A = P from tensor memory, B = the value codes in shared memory (fp16, N-major: token rows as they
//                 lie in the cache), O in tensor memory, fp32.
// Steps of 64 keys leave room for the second S: the scores of step i + 1 are there before the softmax of step i is done,
// and no product waits for another's end.
// Codes turn into fp16 exactly, so the scales of the 16-token blocks never touch the operands: ks goes into the
// exponent's multiplier and vs, as log2 vs, into its offset, one pair for 16 columns; the normaliser takes vs back out
// of each 16-column sum.  log2 vs counts relative to lref, the running maximum over tiles rounded up, and not below
// lref - 60, so that a block of zeros (vs = 0) keeps its place in the normaliser.
//
// Warps 0..7 are the softmax of the two row tiles (thread = row = tensor-memory lane), warps 8..11 fetch codes a tile
// ahead into registers and turn them into fp16 operands, two tiles deep, once for both row tiles; warps 12..15 issue
// the MMAs of S and of O, one product of one row tile each.
//
// Roundings: the weights to fp16 (2^-11; the output is 16-bit; no finer than 2^-33 of the largest value scale, half of
// fp16's last step below 2^(15 - kLazy)), bf16 queries to fp16 after a power of two brought their
// row's largest magnitude to 2^13..2^14 (exact for coordinates within 2^-27 of it).  The running maximum moves only
// when it grows by more than 2^kLazy (weights stay below 2^kLazy, and inside fp16 with the 2^(15 - kLazy) they are
// scaled by), so the output is seldom rescaled, and a tile takes one pass over S: the weights are formed with the
// present maximum and kept in registers until the tile's own maximum is known.
//
// Measured, 4 sequences x 2048 query tokens over up to 8192 keys, 32 / 8 heads, d = 128 (0.96 Tflop): 920-990 us, about
// 1.0 PFLOP/s, 0.60-0.65 of the bf16 GEMM rate.  Nothing is saturated: tensor pipe 55 %, exponentials 55 %, issue slots
// 59 % of the active cycles; without its MMAs, its exponentials or its conversions the kernel is 6-9 % faster each, so
// the chain of hand-overs (a satisfied mbarrier wait costs a warp about 170 clocks) bounds it.  Slower forms: one S of 128
// keys a row tile (1093 us), one issuing warp for all products (1366 us), one a row tile (1024 us), all 64 columns of a
// step loaded at once (1044 us), two threads a row (1124 us).
#pragma once

#include "q8_attend.cuh"
#include "tc.cuh"
#include "warp_mma.cuh"

namespace axr {

constexpr int kPfKeys = 128, kPfStep = 64, kPfThreads = 16 * 32;
constexpr int kLazy = 6;
constexpr float kNoScale = -150.f;  // lref before any positive value scale: below log2 of the smallest, 2^-149

template <int D>
struct PrefillPlan {
  static constexpr uint32_t BLOCK = 128u * 128u;           // a column block: 128 rows x 64 fp16 coordinates (128 bytes)
  static constexpr uint32_t TILE = D / 64 * BLOCK;         // an operand tile: 128 rows x D
  static constexpr uint32_t OFF_Q = 0, OFF_K = 2 * TILE, OFF_V = 4 * TILE;  // two row tiles, two stages each
  static constexpr uint32_t OFF_SC = 6 * TILE;             // [4][32] floats: a key tile's ks[8], off[8], winv[8], lref
  static constexpr uint32_t OFF_BL = OFF_SC + 4 * 32 * 4;  // [4][8] ints: scale blocks of a tile, by converter warp
  static constexpr uint32_t OFF_BAR = OFF_BL + 4 * 8 * 4;
  static constexpr size_t bytes = 1024 + OFF_BAR + 26 * 8;
  static constexpr uint32_t COLS = 512, COL_S = 0, COL_O = 256;  // tensor memory: S of the row tiles, then O, 128 each
  static constexpr int CH = D / 16;                        // 16-byte code chunks of a row
  static constexpr int NL = kPfKeys * CH / 128;            // chunks a converter thread holds of a tile
};

__device__ __forceinline__ float lg2(float x) {  // subnormal x included
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// 16 bytes from global memory, or zeros where !on.  Volatile: the loads stay where they are written, a tile ahead.
__device__ __forceinline__ uint4 load16_if(const uint8_t* p, bool on) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\t"
      "mov.b32 %3, 0;\n\t@p ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"(on ? 1 : 0));
  return v;
}

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Shared-memory matrix descriptor with the 128-byte swizzle.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(lbo >> 4) << 16) |
         (static_cast<uint64_t>(sbo >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// kind::f16, fp16 operands, fp32 accumulation, M = 128; b_mn: B is N-major
__host__ __device__ constexpr uint32_t pf_idesc(int n, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* mbar) {
  const uint32_t mb = static_cast<uint32_t>(__cvta_generic_to_shared(mbar));
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(mb) : "memory");
}

// A bounded wait whose outcome is the same for the whole warp.  Each poll may sleep in hardware for up to a millisecond,
// so that waiting warps leave the issue slots and the shared-memory pipe to the working ones; about two seconds in all.
__device__ __forceinline__ bool warp_wait(uint64_t* mbar, uint32_t parity) {
  const uint32_t mb = static_cast<uint32_t>(__cvta_generic_to_shared(mbar));
  uint32_t done = 0;
  for (int it = 0; it < 2000 && !done; ++it)
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(mb), "r"(parity), "r"(1000000u)
        : "memory");
  return __all_sync(0xffffffffu, done != 0);
}

// Byte offset of the 16-byte chunk j (0..7) of row r in a column block.
__device__ __forceinline__ uint32_t sw128(int r, int j) {
  return static_cast<uint32_t>(r * 128 + ((j ^ (r & 7)) << 4));
}

template <typename T, int D, bool I8>
__global__ void __launch_bounds__(kPfThreads, 1)
q8_prefill_kernel(const __grid_constant__ Q8Attend a, const Q8Tiles tl) {
  using P = PrefillPlan<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw)) & 1023)) & 1023);
  float* sc = reinterpret_cast<float*>(smem + P::OFF_SC);
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + P::OFF_BAR);
  // by stage: operands written, operands read; by row tile and S buffer: S written, weights written, output updated
  uint64_t *k_full = bar, *v_full = bar + 2, *k_free = bar + 4, *v_free = bar + 6;
  uint64_t *s_full = bar + 8, *p_full = bar + 12, *pv_done = bar + 16;  // [row tile][S buffer]
  uint64_t* drain = bar + 20;                                            // [issuing warp], when a wait gave up
  uint32_t* tm_slot = reinterpret_cast<uint32_t*>(bar + 24);
  uint32_t* failed = tm_slot + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // blocks run from the last row tile to the first: with causal rows the later tiles of a sequence are the longer ones
  const int64_t idx = static_cast<int64_t>(gridDim.x) - 1 - blockIdx.x;
  const int split = static_cast<int>(idx % a.splits);
  const int hk = static_cast<int>((idx / a.splits) % a.Hkv);
  const int64_t tile = idx / (static_cast<int64_t>(a.splits) * a.Hkv);
  int b;
  int64_t i0;
  const Q8Span sp = q8_tile_span(a, tl, tile, lane, b, i0);
  if (!q8_tile_live(a, tl, sp, i0, lane)) return;  // uniform over the block
  const int ntok = min(tl.tpt, sp.count - static_cast<int>(i0)), nrow = ntok * a.G;
  const int nq = nrow > 128 ? 2 : 1;                             // row tiles in use
  const int first_lim = sp.pos0 + static_cast<int>(i0) + 1;      // keys the tile's first token sees
  const int begin = split * a.chunk, end = min(min(begin + a.chunk, a.T), first_lim + ntok - 1);
  const int n = end > begin ? (end - begin + kPfKeys - 1) / kPfKeys : 0;  // operand stages
  const int ns = end > begin ? (end - begin + kPfStep - 1) / kPfStep : 0;  // steps

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // a merge may get ready; it waits for this grid's end

  // ---- set-up: barriers, tensor memory, the query operand
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(k_full + i, 128);
      tc::mbar_init(v_full + i, 128);
      tc::mbar_init(k_free + i, nq);
      tc::mbar_init(v_free + i, nq);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(s_full + i, 1);
      tc::mbar_init(p_full + i, 128);
      tc::mbar_init(pv_done + i, 1);
      tc::mbar_init(drain + i, 1);
    }
    *failed = 0;
  }
  if (warp == 12) tc::tmem_alloc(tm_slot, P::COLS);
  float f_row = 0.f;
  int lim = 0;
  int64_t orow = 0;
  if (warp < 8) {
    const int r = threadIdx.x;
    const bool live = r < nrow;
    const int i = static_cast<int>(i0) + (live ? r / a.G : 0), h = hk * a.G + (live ? r % a.G : 0);
    lim = live ? min(first_lim + (i - static_cast<int>(i0)), end) : 0;
    orow = (sp.first + i) * a.Hq + h;
    const T* src = static_cast<const T*>(a.q) + (sp.first + i) * a.q_stride + static_cast<int64_t>(h) * D;
    float mx = 0.f;
    if (live) {
#pragma unroll 4
      for (int c = 0; c < D / 8; ++c) {
        Raw8<T> w;
        float x[8];
        w.load(src + 8 * c);
        w.values(x);
#pragma unroll
        for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(x[e]));
      }
    }
    int ex = 0;
    if (mx > 0.f && isfinite(mx)) frexpf(mx, &ex);
    ex = max(-120, min(114, ex - 14));  // 114: the largest finite queries; -120: 2^-ex stays well inside fp32's range
    const float up = ldexpf(a.mult < 0.f ? -1.f : 1.f, -ex);  // the operand carries the sign, so that f_row >= 0
    f_row = fabsf(a.mult) * ldexpf(1.f, ex);
    if (warp < 4 * nq) {
#pragma unroll 4
      for (int c = 0; c < D / 8; ++c) {
        Raw8<T> w;
        float x[8];
        if (live) w.load(src + 8 * c);
        else w.zero();
        w.values(x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= up;
        store8(reinterpret_cast<__half*>(smem + P::OFF_Q + (r >> 7) * P::TILE + (c >> 3) * P::BLOCK +
                                         sw128(r & 127, c & 7)), x);
      }
    }
    tc::fence_async_smem();
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tm = *tm_slot;
  if (warp >= 8 && warp < 12) {
    if (n > 0) {
    // ---- converters: thread c holds the code chunk (row c / CH + (128 / CH) k, chunk c % CH) of a tile, k < NL
    const int c = threadIdx.x - 256, chunk = c % P::CH, row_c = c / P::CH;
    constexpr int RS = 128 / P::CH;                      // rows between two of a thread's chunks (16 or 32)
    const int32_t* table = a.table + static_cast<size_t>(b) * a.max_blocks;
    const uint8_t* kp = a.kcodes + ((row_c & 15) * D + 16 * chunk);
    const uint8_t* vp = a.vcodes + ((row_c & 15) * D + 16 * chunk);
    uint4 kw[P::NL], vw[P::NL];
    float ks = 0.f, vs = 0.f;
    // lane l: pool scale block (16 rows) of the tile's block l % 8, -1 past the end
    auto blocks_of = [&](int j) {
      int r = -1;
      const int t = begin + j * kPfKeys + 16 * (lane & 7);
      if (t < end) {
        int page = __ldg(table + (t >> a.shift));
        if (page < 0 || page >= a.num_blocks) {
          if (lane < 8) atomicOr(a.status, kStatusBadIndex);
          page = 0;
        }
        r = ((page * a.Hkv + hk) << (a.shift - 4)) + ((t & ((1 << a.shift) - 1)) >> 4);
      }
      return r;
    };
    // the blocks' places, from the lanes that hold them to every thread of the warp
    int* const bl = reinterpret_cast<int*>(smem + P::OFF_BL) + 8 * (warp - 8);
    auto share = [&](int blocks) {
      __syncwarp();
      if (lane < 8) bl[lane] = blocks;
      __syncwarp();
    };
    auto fetch = [&](const uint8_t* codes, uint4 (&w)[P::NL]) {
#pragma unroll
      for (int k = 0; k < P::NL; ++k) {
        const int blk = bl[(row_c + RS * k) >> 4];
        w[k] = load16_if(codes + static_cast<int64_t>(blk) * (16 * D), blk >= 0);
      }
    };
    const int odd = (chunk >> 2) & 1;
    uint8_t* const d0 = smem + (chunk >> 2) * P::BLOCK + sw128(row_c, 2 * (chunk & 3) + odd);
    uint8_t* const d1 = smem + (chunk >> 2) * P::BLOCK + sw128(row_c, 2 * (chunk & 3) + 1 - odd);
    auto convert = [&](uint32_t off, uint4 (&w)[P::NL], int valid) {
      if (valid < kPfKeys) {  // rows no query sees may hold anything (an e4m3 NaN)
#pragma unroll
        for (int k = 0; k < P::NL; ++k)
          if (row_c + RS * k >= valid) w[k] = make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int k = 0; k < P::NL; ++k) {
        // 16 coordinates = two 16-byte chunks; the odd column block stores its second chunk first, so that the eight
        // threads of a row hit eight different banks
        uint4 lo, hi;
        q8_halves<I8>(odd ? w[k].z : w[k].x, lo.x, lo.y);
        q8_halves<I8>(odd ? w[k].w : w[k].y, lo.z, lo.w);
        q8_halves<I8>(odd ? w[k].x : w[k].z, hi.x, hi.y);
        q8_halves<I8>(odd ? w[k].y : w[k].w, hi.z, hi.w);
        *reinterpret_cast<uint4*>(d0 + off + k * (RS * 128)) = lo;
        *reinterpret_cast<uint4*>(d1 + off + k * (RS * 128)) = hi;
      }
    };
    // block table entries run two tiles ahead of the conversion, codes and scales one
    int next = blocks_of(0), after = n > 1 ? blocks_of(1) : -1;
    share(next);
    fetch(kp, kw);
    fetch(vp, vw);
    if (next >= 0) {
      ks = __ldg(a.kscales + next);
      vs = __ldg(a.vscales + next);
    }
    float lref = kNoScale;
    for (int j = 0; j < n; ++j) {
      const int valid = end - begin - j * kPfKeys, st = j & 1;  // rows of the tile that some query sees
      const uint32_t ph = ((j >> 1) - 1) & 1;
      if (j >= 2 && !warp_wait(k_free + st, ph)) { *failed = 1; break; }
      next = after;
      after = j + 2 < n ? blocks_of(j + 2) : -1;
      convert(P::OFF_K + st * P::TILE, kw, valid);
      if (warp == 8) {
        float* scj = sc + (j & 3) * 32;
        const float lv = lg2(vs);
        float top = lv;
#pragma unroll
        for (int x = 4; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        lref = fmaxf(lref, ceilf(top));
        const float off = fmaxf(lv, lref - 60.f) - lref + static_cast<float>(15 - kLazy);
        if (lane < 8) {
          scj[lane] = ks;
          scj[8 + lane] = off;
          scj[16 + lane] = q8_ex2(-off);
        }
        if (lane == 0) scj[24] = lref;
      }
      tc::fence_async_smem();
      tc::mbar_arrive(k_full + st);
      share(next);
      fetch(kp, kw);
      ks = next >= 0 ? __ldg(a.kscales + next) : 0.f;
      vs = next >= 0 ? __ldg(a.vscales + next) : 0.f;
      if (j >= 2 && !warp_wait(v_free + st, ph)) { *failed = 1; break; }
      convert(P::OFF_V + st * P::TILE, vw, valid);
      tc::fence_async_smem();
      tc::mbar_arrive(v_full + st);
      fetch(vp, vw);
    }
    }
  } else if (warp >= 12) {
    // ---- MMA issue: warps 12 and 13 form S of row tiles 0 and 1, warps 14 and 15 their O.  Step i uses S buffer i % 2:
    // its S may be written once the weights of step i - 2, which lie there, have been read (pv_done).  A satisfied wait
    // costs its warp about 170 clocks, so the four chains run side by side and the tensor pipe always has work queued.
    const int q = warp & 1;
    const uint32_t s0 = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    bool ok = true;
    if (q < nq && warp < 14) {
      const uint64_t dq = sw128_desc(s0 + P::OFF_Q + q * P::TILE, 16, 1024);
      for (int i = 0; i < ns; ++i) {
        const int st = (i >> 1) & 1;
        if (!(i & 1) && !(ok = warp_wait(k_full + st, (i >> 2) & 1))) break;
        if (i >= 2 && !(ok = warp_wait(pv_done + 2 * q + (i & 1), ((i >> 1) - 1) & 1))) break;
        tc::fence_after();
        const uint64_t dk = sw128_desc(s0 + P::OFF_K + st * P::TILE + (i & 1) * (kPfStep * 128), 16, 1024);
        if (elect_one()) {
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            const uint32_t o = ((s >> 2) * P::BLOCK + (s & 3) * 32u) >> 4;
            mma_ss(tm + P::COL_S + 128 * q + kPfStep * (i & 1), dq + o, dk + o, pf_idesc(kPfStep, false), s > 0);
          }
          mma_commit(s_full + 2 * q + (i & 1));
          if (i & 1) mma_commit(k_free + st);
        }
        __syncwarp();
      }
    } else if (q < nq) {
      for (int i = 0; i < ns; ++i) {
        const int st = (i >> 1) & 1;
        if (!(i & 1) && !(ok = warp_wait(v_full + st, (i >> 2) & 1))) break;
        if (!(ok = warp_wait(p_full + 2 * q + (i & 1), (i >> 1) & 1))) break;
        tc::fence_after();
        const uint64_t dv = sw128_desc(s0 + P::OFF_V + st * P::TILE + (i & 1) * (kPfStep * 128), P::BLOCK, 1024);
        if (elect_one()) {
#pragma unroll
          for (int s = 0; s < kPfStep / 16; ++s)
            mma_ts(tm + P::COL_O + 128 * q, tm + P::COL_S + 128 * q + kPfStep * (i & 1) + 8 * s, dv + s * (2048u >> 4),
                   pf_idesc(D, true), i > 0 || s > 0);
          mma_commit(pv_done + 2 * q + (i & 1));
          if (i & 1) mma_commit(v_free + st);
        }
        __syncwarp();
      }
    }
    if (!ok) {
      // a wait gave up: let the products issued so far end, bounded again, before tensor memory is freed
      *failed = 1;
      if (elect_one()) mma_commit(drain + (warp - 12));
      __syncwarp();
      warp_wait(drain + (warp - 12), 0);
    }
  } else {
    if (warp < 4 * nq) {
    // ---- softmax: thread = row
    const int q = warp >> 2;
    const uint32_t tq = tm + (static_cast<uint32_t>((warp & 3) * 32) << 16) + P::COL_S + 128 * q;
    const uint32_t to = tm + (static_cast<uint32_t>((warp & 3) * 32) << 16) + P::COL_O + 128 * q;
    float m = threadIdx.x < nrow ? -INFINITY : 0.f, l = 0.f, lref = kNoScale;  // rows not in use never ask for a second pass
    bool ok = true;
    // 16 columns of weights from 16 of S: 2^(s cc + off - m), packed to fp16; returns their sum
    auto weights = [&](const uint32_t (&x)[16], float cc, float off, uint32_t (&w)[8]) {
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const float2 y = fma2(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), make_float2(cc, cc),
                              make_float2(off, off));
        const float2 p = make_float2(q8_ex2(y.x), q8_ex2(y.y));
        sum = add2(sum, p);
        w[e >> 1] = pack_h2(p.x, p.y);
      }
      return sum.x + sum.y;
    };
    for (int i = 0; i < ns; ++i) {
      if (!(ok = warp_wait(s_full + 2 * q + (i & 1), (i >> 1) & 1))) break;
      tc::fence_after();
      const float* scj = sc + ((i >> 1) & 3) * 32 + (i & 1) * (kPfStep / 16);  // the step's ks; off and winv 8 and 16 on
      const float top = sc[((i >> 1) & 3) * 32 + 24];
      const uint32_t ts = tq + kPfStep * (i & 1);
      const int t1 = begin + (i + 1) * kPfStep;
      const bool masked = t1 > first_lim || t1 > end;      // some column is hidden from some row; uniform
      uint32_t w[kPfStep / 16][8];
      float mx = -INFINITY, lt = 0.f;
      bool again = masked || top != lref;              // uniform
      if (!again) {
        // one pass: the weights with the maximum so far, the tile's own maximum beside them
        uint32_t x[2][16];
        tc::ld_x16(ts, x[0]);
#pragma unroll
        for (int k = 0; k < kPfStep / 16; ++k) {
          tc::wait_ld();
          if (k + 1 < kPfStep / 16) tc::ld_x16(ts + 16 * (k + 1), x[(k + 1) & 1]);
          const float cc = scj[k] * f_row;
          float y = __uint_as_float(x[k & 1][0]);
#pragma unroll
          for (int e = 1; e < 15; e += 2) y = max3(y, __uint_as_float(x[k & 1][e]), __uint_as_float(x[k & 1][e + 1]));
          mx = max3(mx, y * cc, __uint_as_float(x[k & 1][15]) * cc);
          lt = fmaf(weights(x[k & 1], cc, scj[8 + k] - m, w[k]), scj[16 + k], lt);
        }
        again = __any_sync(0xffffffffu, !(mx <= m + static_cast<float>(kLazy)));
      }
      if (again) {
        // the maximum of the visible columns first; the output is rescaled when it, or lref, moves
        const int vis = lim - (t1 - kPfStep);              // columns below vis are visible
        mx = -INFINITY;
#pragma unroll 1
        for (int k = 0; k < kPfStep / 16; ++k) {
          uint32_t x[16];
          tc::ld_x16(ts + 16 * k, x);
          tc::wait_ld();
          const float cc = scj[k] * f_row;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            mx = fmaxf(mx, 16 * k + e < vis ? __uint_as_float(x[e]) * cc : -INFINITY);
        }
        float alpha = 1.f;
        if (mx > m + static_cast<float>(kLazy)) {          // m = -inf: any finite maximum
          alpha = m == -INFINITY ? 0.f : q8_ex2(m - mx);
          m = mx;
        }
        l *= alpha;
        alpha *= q8_ex2(lref - top);
        lref = top;
        if (i > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          if (!(ok = warp_wait(pv_done + 2 * q + ((i - 1) & 1), ((i - 1) >> 1) & 1))) break;
          tc::fence_after();
#pragma unroll 1
          for (int k = 0; k < D / 16; ++k) {
            uint32_t o[16];
            tc::ld_x16(to + 16 * k, o);
            tc::wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tc::st_x16(to + 16 * k, o);
          }
        }
        const float mm = m == -INFINITY ? 0.f : m;
        lt = 0.f;
#pragma unroll
        for (int k = 0; k < kPfStep / 16; ++k) {
          uint32_t x[16];
          tc::ld_x16(ts + 16 * k, x);
          tc::wait_ld();
          const float cc = scj[k] * f_row;
          // a hidden column becomes -inf, whatever its scale: the multiplier is 1 where it is not positive
          const float c1 = cc > 0.f ? cc : 1.f, c0 = cc > 0.f ? 1.f : 0.f;
#pragma unroll
          for (int e = 0; e < 16; ++e)
            x[e] = 16 * k + e < vis ? __float_as_uint(__uint_as_float(x[e]) * c0) : 0xff800000u;
          lt = fmaf(weights(x, c1, scj[8 + k] - mm, w[k]), scj[16 + k], lt);
        }
      }
      l += lt;
#pragma unroll
      for (int k = 0; k < kPfStep / 32; ++k) {
        uint32_t y[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = w[2 * k + (e >> 3)][e & 7];
        tc::st_x16(ts + 16 * k, y);
      }
      tc::wait_st();
      tc::fence_before();
      tc::mbar_arrive(p_full + 2 * q + (i & 1));
    }
    if (ok && ns > 0) {
      ok = warp_wait(pv_done + 2 * q + ((ns - 1) & 1), ((ns - 1) >> 1) & 1);
      tc::fence_after();
    }
    if (!ok) *failed = 1;
    const bool live = threadIdx.x < nrow;
    const float nan = __uint_as_float(0x7fc00000u);
    // times 2^lref in two factors (one could leave fp32's normal range), times 2^-(15 - kLazy), over l; NaN stays
    const float half = floorf(0.5f * lref), f2 = q8_ex2(lref - half);
    const float f1 = q8_ex2(half - static_cast<float>(15 - kLazy)) / (a.splits == 1 && l != 0.f ? l : 1.f);
    const int64_t part = orow * a.splits + split;
#pragma unroll 1
    for (int k = 0; k < D / 16; ++k) {
      uint32_t o[16];
      float x[16];
      if (ok && n > 0) {
        tc::ld_x16(to + 16 * k, o);
        tc::wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = l == 0.f ? 0.f : __uint_as_float(o[e]) * f1 * f2;
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = ok ? 0.f : nan;
      }
      if (live) {
        float y[2][8];
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e >> 3][e & 7] = x[e];
        if (a.splits == 1) {
          T* dst = static_cast<T*>(a.out) + orow * D + 16 * k;
          store8(dst, y[0]);
          store8(dst + 8, y[1]);
        } else {
          float* dst = a.ws_o + part * D + 16 * k;
          store8(dst, y[0]);
          store8(dst + 8, y[1]);
        }
      }
    }
    if (live && a.splits > 1) {
      a.ws_m[part] = m;
      a.ws_l[part] = ok ? l : nan;
    }
    }
  }
  tc::fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *failed) atomicOr(a.status, 1u);
  if (warp == 12) {
    tc::fence_after();
    tc::tmem_dealloc(tm, P::COLS);
  }
}

}  // namespace axr
