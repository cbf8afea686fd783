// Attention of many query tokens over the paged 8-bit cache on the tcgen05 tensor cores.
//
// One thread block takes a row tile of up to 128 query rows (tokens x heads of one KV head's group) and a range of the
// token axis, in key tiles of 128 tokens:
//   S = Q K^T     M = 128 rows, N = 128 tokens: Q and the key codes in shared memory (fp16, K-major, 128-byte swizzle),
//                 S in tensor memory, fp32;
//   P = 2^(ks f S - m), times vs / vref, rounded to fp16 and stored over S in tensor memory;
//   O += P V      A = P from tensor memory, B = the value codes in shared memory (fp16, N-major: token rows as they
//                 lie in the cache), O in tensor memory, fp32.
// Codes turn into fp16 exactly, so the scales of the 16-token blocks never touch the operands: ks goes into the
// exponent's multiplier and vs onto the weights, one factor for 16 columns.
//
// Warps 0..3 are the softmax (thread = row = tensor-memory lane), warps 4..7 fetch codes two tiles ahead into registers
// and turn them into fp16 shared-memory operands, warp 8 issues the MMAs.  Two thread blocks share an SM (256 of its 512
// tensor-memory columns and 97 KB of shared memory each), so that one's MMAs run under the other's softmax.
//
// Roundings: the weights to fp16 (2^-11; the output is 16-bit), bf16 queries to fp16 after a power of two brought their
// row's largest magnitude to 2^13..2^14 (exact for coordinates within 2^-27 of it).  The running maximum moves only
// when it grows by more than 2^kLazy (weights stay below 2^kLazy, and inside fp16 with the 2^(15 - kLazy) they are
// scaled by), so the output is seldom rescaled.
#pragma once

#include "q8_attend.cuh"
#include "tc.cuh"

namespace axr {

constexpr int kPfRows = 128, kPfKeys = 128, kPfThreads = 288;
constexpr int kLazy = 6;
constexpr float kPfUp = static_cast<float>(1 << (15 - kLazy));

template <int D>
struct PrefillPlan {
  static constexpr int CB = D / 64;                        // 64-coordinate column blocks of 128-byte rows
  static constexpr uint32_t BLOCK = 128u * 128u;           // bytes of one column block: 128 rows x 128 bytes
  static constexpr uint32_t OFF_Q = 0, OFF_K = CB * BLOCK, OFF_V = 2 * CB * BLOCK;
  static constexpr uint32_t OFF_SC = 3 * CB * BLOCK;       // [2][16] floats: ks, vs of a tile's 8 scale blocks
  static constexpr uint32_t OFF_BAR = OFF_SC + 2 * 16 * 4;
  static constexpr size_t bytes = 1024 + OFF_BAR + 64;
  static constexpr int COLS = 256, COL_S = 0, COL_O = 128; // tensor memory
  static constexpr int CH = D / 16;                        // 16-byte code chunks of a row
  static constexpr int NL = kPfKeys * CH / 128;            // chunks a converter thread holds of a tile
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long rd;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(rd)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return *reinterpret_cast<float2*>(&rd);
}

__device__ __forceinline__ void tm_ld32(uint32_t taddr, float (&d)[32]) {
  uint32_t* u = reinterpret_cast<uint32_t*>(d);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]),
        "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]), "=r"(u[16]),
        "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]), "=r"(u[24]),
        "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
      : "r"(taddr)
      : "memory");
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

// A bounded wait whose outcome is the same for the whole warp.
__device__ __forceinline__ bool warp_wait(uint64_t* mbar, uint32_t parity) {
  return __all_sync(0xffffffffu, tc::mbar_wait(mbar, parity));
}

// Byte offset of the 16-byte chunk j (0..7) of row r in a column block.
__device__ __forceinline__ uint32_t sw128(int r, int j) {
  return static_cast<uint32_t>(r * 128 + ((j ^ (r & 7)) << 4));
}

template <typename T, int D, bool I8>
__global__ void __launch_bounds__(kPfThreads, 2)
q8_prefill_kernel(const __grid_constant__ Q8Attend a, const Q8Tiles tl) {
  using P = PrefillPlan<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (static_cast<uint32_t>(__cvta_generic_to_shared(smem_raw)) & 1023)) & 1023);
  float* sc = reinterpret_cast<float*>(smem + P::OFF_SC);
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + P::OFF_BAR);
  uint64_t *k_full = bar, *v_full = bar + 1, *p_full = bar + 2, *qk_done = bar + 3, *pv_done = bar + 4;
  uint32_t* tm_slot = reinterpret_cast<uint32_t*>(bar + 5);
  uint32_t* failed = tm_slot + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // blocks run from the last row tile to the first: with causal rows the later tiles of a sequence are the longer ones
  const int64_t idx = static_cast<int64_t>(gridDim.x) - 1 - blockIdx.x;
  const int split = static_cast<int>(idx % a.splits);
  const int hk = static_cast<int>((idx / a.splits) % a.Hkv);
  const int64_t tile = idx / (static_cast<int64_t>(a.splits) * a.Hkv);
  int b;
  int64_t i0;
  q8_tile(a, tl, tile, lane, b, i0);
  const Q8Span sp = q8_span(a, b);
  if (!q8_tile_live(a, tl, sp, i0, lane)) return;  // uniform over the block
  const int ntok = min(tl.tpt, sp.count - static_cast<int>(i0)), nrow = ntok * a.G;
  const int first_lim = sp.pos0 + static_cast<int>(i0) + 1;      // keys the tile's first token sees
  const int begin = split * a.chunk, end = min(begin + a.chunk, first_lim + ntok - 1);
  const int n = end > begin ? (end - begin + kPfKeys - 1) / kPfKeys : 0;

  // ---- set-up: barriers, tensor memory, the query operand
  if (threadIdx.x == 0) {
    tc::mbar_init(k_full, 128);
    tc::mbar_init(v_full, 128);
    tc::mbar_init(p_full, 128);
    tc::mbar_init(qk_done, 1);
    tc::mbar_init(pv_done, 1);
    *failed = 0;
  }
  if (warp == 8) tc::tmem_alloc(tm_slot, P::COLS);
  float f_row = 0.f;
  int lim = 0;
  int64_t orow = 0;
  if (warp < 4) {
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
    ex = max(-100, min(100, ex - 14));
    const float up = ldexpf(a.mult < 0.f ? -1.f : 1.f, -ex);  // the operand carries the sign, so that f_row >= 0
    f_row = fabsf(a.mult) * ldexpf(1.f, ex);
#pragma unroll 4
    for (int c = 0; c < D / 8; ++c) {
      Raw8<T> w;
      float x[8];
      if (live) w.load(src + 8 * c);
      else w.zero();
      w.values(x);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= up;
      store8(reinterpret_cast<__half*>(smem + P::OFF_Q + (c >> 3) * P::BLOCK + sw128(r, c & 7)), x);
    }
    tc::fence_async_smem();
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tm = *tm_slot;

  if (warp >= 4 && warp < 8 && n > 0) {
    // ---- converters: thread c holds the code chunk (row c / CH + (128 / CH) k, chunk c % CH) of a tile, k < NL
    const int c = threadIdx.x - 128, chunk = c % P::CH, row_c = c / P::CH;
    constexpr int RS = 128 / P::CH;                      // rows between two of a thread's chunks (16 or 32)
    const int32_t* table = a.table + static_cast<size_t>(b) * a.max_blocks;
    uint4 kw[P::NL], vw[P::NL];
    float ks = 0.f, vs = 0.f;
    // lane l < 8: pool row of scale block l of a tile, -1 past the end
    auto rows_of = [&](int j) {
      int64_t r = -1;
      const int t = begin + j * kPfKeys + 16 * (lane & 7);
      if (t < end) {
        int page = __ldg(table + (t >> a.shift));
        if (page < 0 || page >= a.num_blocks) {
          if (lane < 8) atomicOr(a.status, kStatusBadIndex);
          page = 0;
        }
        r = ((static_cast<int64_t>(page) * a.Hkv + hk) << a.shift) + (t & ((1 << a.shift) - 1));
      }
      return r;
    };
    auto fetch = [&](const uint8_t* codes, int64_t rows, uint4 (&w)[P::NL]) {
#pragma unroll
      for (int k = 0; k < P::NL; ++k) {
        const int r = row_c + RS * k;
        const int64_t base = __shfl_sync(0xffffffffu, rows, r >> 4);
        w[k] = base >= 0 ? __ldg(reinterpret_cast<const uint4*>(codes + (base + (r & 15)) * D) + chunk)
                         : make_uint4(0, 0, 0, 0);
      }
    };
    auto convert = [&](uint32_t off, const uint4 (&w)[P::NL], int valid) {
#pragma unroll
      for (int k = 0; k < P::NL; ++k) {
        const int r = row_c + RS * k;
        uint4 x = w[k];
        if (r >= valid) x = make_uint4(0, 0, 0, 0);
        uint4 lo, hi;
        q8_halves<I8>(x.x, lo.x, lo.y);
        q8_halves<I8>(x.y, lo.z, lo.w);
        q8_halves<I8>(x.z, hi.x, hi.y);
        q8_halves<I8>(x.w, hi.z, hi.w);
        // 16 coordinates = two 16-byte chunks; the odd column block stores its second chunk first, so that the eight
        // threads of a row hit eight different banks
        uint8_t* dst = smem + off + (chunk >> 2) * P::BLOCK;
        const int j0 = 2 * (chunk & 3), odd = (chunk >> 2) & 1;
        *reinterpret_cast<uint4*>(dst + sw128(r, j0 + odd)) = odd ? hi : lo;
        *reinterpret_cast<uint4*>(dst + sw128(r, j0 + 1 - odd)) = odd ? lo : hi;
      }
    };
    int64_t rows = rows_of(0);
    fetch(a.kcodes, rows, kw);
    fetch(a.vcodes, rows, vw);
    if (rows >= 0) {
      ks = __ldg(a.kscales + (rows >> 4));
      vs = __ldg(a.vscales + (rows >> 4));
    }
    for (int j = 0; j < n; ++j) {
      const int valid = end - begin - j * kPfKeys;       // rows of the tile that some query sees
      const int64_t next = j + 1 < n ? rows_of(j + 1) : -1;
      if (j > 0 && !warp_wait(qk_done, (j - 1) & 1)) { *failed = 1; break; }
      convert(P::OFF_K, kw, valid);
      if (c < 8) {
        sc[(j & 1) * 16 + c] = ks;
        sc[(j & 1) * 16 + 8 + c] = vs;
      }
      tc::fence_async_smem();
      tc::mbar_arrive(k_full);
      ks = vs = 0.f;
      if (next >= 0) {
        ks = __ldg(a.kscales + (next >> 4));
        vs = __ldg(a.vscales + (next >> 4));
      }
      fetch(a.kcodes, next, kw);
      if (j > 0 && !warp_wait(pv_done, (j - 1) & 1)) { *failed = 1; break; }
      convert(P::OFF_V, vw, valid);
      tc::fence_async_smem();
      tc::mbar_arrive(v_full);
      fetch(a.vcodes, next, vw);
    }
  } else if (warp == 8 && n > 0) {
    // ---- MMA issue
    if (lane == 0) {
      const uint32_t s0 = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
      for (int j = 0; j < n; ++j) {
        if (!tc::mbar_wait(k_full, j & 1) || (j > 0 && !tc::mbar_wait(pv_done, (j - 1) & 1))) { *failed = 1; break; }
        tc::fence_after();
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint32_t o = (s >> 2) * P::BLOCK + (s & 3) * 32u;
          mma_ss(tm + P::COL_S, sw128_desc(s0 + P::OFF_Q + o, 16, 1024), sw128_desc(s0 + P::OFF_K + o, 16, 1024),
                 pf_idesc(kPfKeys, false), s > 0);
        }
        mma_commit(qk_done);
        if (!tc::mbar_wait(v_full, j & 1) || !tc::mbar_wait(p_full, j & 1)) { *failed = 1; break; }
        tc::fence_after();
#pragma unroll
        for (int s = 0; s < kPfKeys / 16; ++s)
          mma_ts(tm + P::COL_O, tm + P::COL_S + 8 * s, sw128_desc(s0 + P::OFF_V + s * 2048u, P::BLOCK, 1024),
                 pf_idesc(D, true), j > 0 || s > 0);
        mma_commit(pv_done);
      }
    }
  } else if (warp < 4) {
    // ---- softmax: thread = row
    const uint32_t ts = tm + (static_cast<uint32_t>(warp * 32) << 16) + P::COL_S;
    const uint32_t to = tm + (static_cast<uint32_t>(warp * 32) << 16) + P::COL_O;
    float m = -INFINITY, vref = 0.f;
    float2 l2 = make_float2(0.f, 0.f);
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      if (!warp_wait(qk_done, j & 1)) { ok = false; break; }
      tc::fence_after();
      const int t0 = begin + j * kPfKeys;
      const bool masked = t0 + kPfKeys > first_lim || t0 + kPfKeys > end;  // uniform
      const float* scj = sc + (j & 1) * 16;
      float cs[8], vmax = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        cs[i] = scj[i] * f_row;
        vmax = fmaxf(vmax, scj[8 + i]);
      }
      const int vis = lim - t0;                            // columns below vis are visible
      float mx = -INFINITY;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float s[32];
        tm_ld32(ts + 32 * k, s);
        tc::wait_ld();
        if (masked) {
#pragma unroll
          for (int e = 0; e < 32; ++e) mx = fmaxf(mx, 32 * k + e < vis ? s[e] * cs[2 * k + (e >> 4)] : -INFINITY);
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float q = s[16 * h];
#pragma unroll
            for (int e = 1; e < 16; ++e) q = fmaxf(q, s[16 * h + e]);
            mx = fmaxf(mx, q * cs[2 * k + h]);
          }
        }
      }
      // the reference maximum and value scale; the output is rescaled when either moves
      float alpha = 1.f;
      if (mx > m + static_cast<float>(kLazy)) {            // m = -inf: any finite maximum
        alpha = m == -INFINITY ? 0.f : ex2(m - mx);
        m = mx;
      }
      float beta = 1.f;
      if (vmax > vref) {                                   // uniform
        const float up = __uint_as_float((__float_as_uint(vmax) + 0x7fffffu) & 0x7f800000u);
        beta = vref / up;
        vref = up;
      }
      l2.x *= alpha;
      l2.y *= alpha;
      alpha *= beta;
      if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
        if (!warp_wait(pv_done, (j - 1) & 1)) { ok = false; break; }
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
      const float vf = vref > 0.f ? kPfUp / vref : 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float s[32];
        uint32_t w[16];
        tm_ld32(ts + 32 * k, s);
        tc::wait_ld();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float cc = cs[2 * k + h], vv = scj[8 + 2 * k + h] * vf;
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const int col = 16 * h + e;
            float x0 = fmaf(s[col], cc, -mm), x1 = fmaf(s[col + 1], cc, -mm);
            if (masked) {
              x0 = 32 * k + col < vis ? x0 : -INFINITY;
              x1 = 32 * k + col + 1 < vis ? x1 : -INFINITY;
            }
            float2 p = make_float2(ex2(x0), ex2(x1));
            l2 = add2(l2, p);
            p = mul2(p, make_float2(vv, vv));
            const __half2 hp = __floats2half2_rn(p.x, p.y);
            w[(col) >> 1] = *reinterpret_cast<const uint32_t*>(&hp);
          }
        }
        tc::st_x16(ts + 16 * k, w);
      }
      tc::wait_st();
      tc::fence_before();
      tc::mbar_arrive(p_full);
    }
    if (ok && n > 0) {
      ok = warp_wait(pv_done, (n - 1) & 1);
      tc::fence_after();
    }
    if (!ok) *failed = 1;
    const float l = l2.x + l2.y;
    const bool live = threadIdx.x < nrow;
    const float nan = __uint_as_float(0x7fc00000u);
    const float unscale = vref * (1.f / kPfUp);
    const float f = a.splits == 1 ? (l > 0.f ? unscale / l : 0.f) : unscale;
    const int64_t part = ((tile * a.Hkv + hk) * kPfRows + threadIdx.x) * a.splits + split;
#pragma unroll 1
    for (int k = 0; k < D / 16; ++k) {
      uint32_t o[16];
      float x[16];
      if (ok && n > 0) {
        tc::ld_x16(to + 16 * k, o);
        tc::wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = l > 0.f ? __uint_as_float(o[e]) * f : 0.f;
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = ok ? 0.f : nan;
      }
      if (live) {
        if (a.splits == 1) {
          T* dst = static_cast<T*>(a.out) + orow * D + 16 * k;
          store8(dst, *reinterpret_cast<float(*)[8]>(x));
          store8(dst + 8, *reinterpret_cast<float(*)[8]>(x + 8));
        } else {
          float* dst = a.ws_o + part * D + 16 * k;
          store8(dst, *reinterpret_cast<float(*)[8]>(x));
          store8(dst + 8, *reinterpret_cast<float(*)[8]>(x + 8));
        }
      }
    }
    if (live && a.splits > 1) {
      a.ws_m[part] = m;
      a.ws_l[part] = ok ? l : nan;
    }
  }
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *failed) atomicOr(a.status, 1u);
  if (warp == 8) {
    tc::fence_after();
    tc::tmem_dealloc(tm, P::COLS);
  }
}

}  // namespace axr
