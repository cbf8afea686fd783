// Decode attention over the paged 8-bit cache: every warp is a worker on an equal share of the batch's key tiles.
//
// The work is a flat sequence of 32-token key tiles: sequence after sequence, for each of its row tiles (up to 8 NRG
// query rows: tokens x heads of the group) and KV heads, the tiles of that sequence's length.  Worker w takes tiles
// [w S, (w + 1) S), S = ceil(total / workers) but at least kDecMinTiles, whatever units (row tile x KV head) they fall
// into: lengths in the batch need not be alike, and nothing of the split depends on what the host knows.  A unit that
// lies inside one share is finished there; a unit cut by a share's edge leaves a partial (m, l, o) in the share's slot
// 0 (the unit the share begins in) or 1 (a later one), merged by q8_merge_kernel.
//
// A worker streams its tiles through a ring of its own: TMA boxes of 16 or 32 token rows (a pool block may end inside
// a tile only at bt = 16), swizzled, each completing on the stage's mbarrier.  Block-table entries and scales of 32
// tiles sit in the lanes' registers, fetched half a batch ahead.
//
// Both products run as mma.sync.m16n8k16 on fp16 operands with the query rows as the N side, so that no half of a tile
// is empty for 8 rows:
//   S^T = K Q^T    A = 16 tokens x 16 coordinates of codes, B = the queries;
//   O^T += V^T P^T A = 16 coordinates x 16 tokens of codes, B = the weights, transposed in registers (movmatrix).
// The codes enter exactly; queries as PQ fp16 planes, hi and lo (about 22 bits) for fp32, one for 16-bit types, which a
// power of two makes exact; softmax weights as PP planes, one for bf16 (a rounding to 2^-11, where the output's is 2^-9),
// hi and lo for fp16 and fp32; no plane holds less than 2^-24, so a token's value is within 2^-38 of the largest scale.
// Coordinates and tokens may be summed in any order, so each lane reads 16-byte runs of a code row: of the key rows
// 8 n + g the bytes [D/4 t, D/4 t + D/4), whose word s feeds k-step s; of the value rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9
// (+ 16) the bytes [D/8 g, D/8 g + D/8), bytes 2 j and 2 j + 1 going to rows g and g + 8 of coordinate tile j.  Every
// code is read from shared memory once, by 128-bit loads that the swizzle keeps free of bank conflicts.
// (tcgen05 would need the codes as fp16 in shared memory, four times this traffic, for 4 to 16 query rows of 128.)
//
// HBM bounds long calls: 8 sequences x 32768 tokens, 32 / 8 heads, d = 128 take 94-103 us with the merge, 5.2-5.7 TB/s
// or 0.80-0.87 of the copy rate; the same batch with 16 query heads per KV head (two row
// groups) is bound by issue slots.  Small calls are a chain of round trips: lengths, block table, tiles, partials (one
// sequence of 4096 tokens: 12 us, 8 without the merge).  With the query rows as the M side, hi and lo planes stacked in
// one tile, the long call took 121 us: twice the MMAs and accumulators, eight warps instead of twelve.
#pragma once

#include <cuda.h>

#include <type_traits>

#include "dense_stream.cuh"
#include "q8_merge.cuh"

namespace axr {

constexpr int kDecTile = 32;      // tokens per tile
constexpr int kDecMinTiles = 2;   // smallest share

// Twelve warps of 168 registers hold one row group without spilling, eight of 255 two; the rings fill shared memory.
template <int D, int NRG>
struct DecodePlan {
  static constexpr int WARPS = q8_decode_warps(NRG);
  static constexpr int NS = NRG == 1 ? 2 : 3;               // stages per warp
  static constexpr size_t PLANE = kDecTile * D;             // the K (or V) codes of a stage
  static constexpr size_t STAGE = 2 * PLANE;
  static constexpr size_t OFF_MBAR = WARPS * NS * STAGE;
  static constexpr size_t bytes = 1024 + OFF_MBAR + WARPS * NS * 8;
};

// 8-bit codes of two rows, 4 coordinates each, as 4 half2 (row a's coordinate, row b's coordinate)
template <bool I8>
__device__ __forceinline__ void q8_pairs(uint32_t a, uint32_t b, uint32_t (&h)[4]) {
  q8_halves<I8>(__byte_perm(a, b, 0x5140), h[0], h[1]);
  q8_halves<I8>(__byte_perm(a, b, 0x7362), h[2], h[3]);
}

// Byte offset in a plane of the 16-byte chunk c of row r: the TMA swizzles of 128-byte and 64-byte rows.
template <int D>
__device__ __forceinline__ uint32_t q8_swz(int r, int c) {
  if constexpr (D == 128) return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4));
  else return static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// Quotient of non-negative values: 32-bit division where both fit (a 64-bit one takes about a hundred instructions).
__device__ __forceinline__ int64_t q8_div(int64_t x, int64_t y) {
  if (((x | y) >> 32) == 0) return static_cast<uint32_t>(x) / static_cast<uint32_t>(y);
  return x / y;
}

// Row tiles and key tiles of a sequence.
struct Q8Extent {
  int rts;    // row tiles
  int tiles;  // key tiles of each (those of its last row tile)
};
__device__ __forceinline__ Q8Extent q8_extent(const Q8Attend& a, const Q8Tiles& tl, const Q8Span& sp) {
  Q8Extent e;
  e.rts = tl.one ? (sp.count > 0 && sp.count <= tl.tpt ? 1 : 0) : (sp.count + tl.tpt - 1) / tl.tpt;
  e.tiles = e.rts > 0 ? (sp.keys(a.T) + kDecTile - 1) / kDecTile : 0;
  return e;
}

// A sequence in the flat tile sequence.
struct Q8Place {
  int b;
  int64_t begin;  // its first tile
  Q8Span sp;
  Q8Extent ext;
};

// The flat tile sequence as a warp holds it: lane l has sequences l and 32 + l (their entries read once, in one round
// trip); batches of more than 64 sequences are read again by each search.
struct Q8Flat {
  Q8Span sp[2];
  Q8Extent ext[2];
  int64_t ex[2], n[2];  // tiles before, tiles of
  int64_t total;

  __device__ __forceinline__ static void scan(const Q8Attend& a, const Q8Tiles& tl, int lane, int b0, int64_t& sum,
                                              Q8Span& sp, Q8Extent& e, int64_t& ex, int64_t& n) {
    const bool on = b0 + lane < a.B;
    sp = q8_span(a, on ? b0 + lane : 0);
    e = q8_extent(a, tl, sp);
    n = on ? static_cast<int64_t>(e.rts) * a.Hkv * e.tiles : 0;
    int64_t inc = n;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, inc, m);
      if (lane >= m) inc += o;
    }
    ex = sum + inc - n;
    sum += __shfl_sync(0xffffffffu, inc, 31);
  }

  __device__ __forceinline__ void load(const Q8Attend& a, const Q8Tiles& tl, int lane) {
    total = 0;
    scan(a, tl, lane, 0, total, sp[0], ext[0], ex[0], n[0]);
    n[1] = 0;
    if (a.B > 32) scan(a, tl, lane, 32, total, sp[1], ext[1], ex[1], n[1]);
    for (int b0 = 64; b0 < a.B; b0 += 32) {
      Q8Span s;
      Q8Extent e;
      int64_t x, y;
      scan(a, tl, lane, b0, total, s, e, x, y);
    }
  }

  __device__ __forceinline__ static void take(Q8Place& r, const Q8Span& sp, const Q8Extent& e, int64_t ex, int b0,
                                              int src) {
    r.b = b0 + src;
    r.begin = __shfl_sync(0xffffffffu, ex, src);
    r.sp.first = __shfl_sync(0xffffffffu, sp.first, src);
    r.sp.count = __shfl_sync(0xffffffffu, sp.count, src);
    r.sp.pos0 = __shfl_sync(0xffffffffu, sp.pos0, src);
    r.ext.rts = __shfl_sync(0xffffffffu, e.rts, src);
    r.ext.tiles = __shfl_sync(0xffffffffu, e.tiles, src);
  }

  // The sequence that holds flat tile x < total.
  __device__ __forceinline__ Q8Place at_tile(const Q8Attend& a, const Q8Tiles& tl, int lane, int64_t x) const {
    const auto pick = [=](int64_t ex_, int64_t n_) { return ex_ <= x && x < ex_ + n_; };
    Q8Place r;
    unsigned who = __ballot_sync(0xffffffffu, pick(ex[0], n[0]));
    if (who) {
      take(r, sp[0], ext[0], ex[0], 0, __ffs(who) - 1);
      return r;
    }
    who = __ballot_sync(0xffffffffu, a.B > 32 && pick(ex[1], n[1]));
    if (who) {
      take(r, sp[1], ext[1], ex[1], 32, __ffs(who) - 1);
      return r;
    }
    int64_t sum = __shfl_sync(0xffffffffu, ex[1] + n[1], 31);  // tiles of the first 64
    for (int b0 = 64; b0 < a.B; b0 += 32) {
      Q8Span s;
      Q8Extent e;
      int64_t x0, y;
      scan(a, tl, lane, b0, sum, s, e, x0, y);
      who = __ballot_sync(0xffffffffu, pick(x0, y));
      if (who) {
        take(r, s, e, x0, b0, __ffs(who) - 1);
        return r;
      }
    }
    r.b = 0;
    r.begin = 0;
    r.sp = {0, 0, 0};
    r.ext = {0, 1};
    return r;
  }
};

__device__ __forceinline__ int64_t q8_warp_sum(int64_t v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// Sequence b in the flat tile sequence, and the tiles of all: sums instead of a search where b is known.
__device__ __forceinline__ Q8Place q8_place(const Q8Attend& a, const Q8Tiles& tl, int lane, int b, int64_t& total) {
  int64_t all = 0, before = 0;
  Q8Span own{0, 0, 0};  // sequence b's, in lane b % 32
#pragma unroll 2
  for (int c = lane; c < a.B; c += 32) {
    const Q8Span sp = q8_span<false>(a, c);
    const Q8Extent e = q8_extent(a, tl, sp);
    const int64_t n = static_cast<int64_t>(e.rts) * a.Hkv * e.tiles;
    all += n;
    before += c < b ? n : 0;
    if (c == b) own = sp;
  }
  total = q8_warp_sum(all);
  Q8Place r;
  r.b = b;
  r.begin = q8_warp_sum(before);
  r.sp.first = __shfl_sync(0xffffffffu, own.first, b & 31);
  r.sp.count = __shfl_sync(0xffffffffu, own.count, b & 31);
  r.sp.pos0 = __shfl_sync(0xffffffffu, own.pos0, b & 31);
  r.ext = q8_extent(a, tl, r.sp);
  return r;
}

__device__ __forceinline__ int64_t q8_share(int64_t total, int workers) {
  const int64_t s = q8_div(total + workers - 1, workers);
  return s > kDecMinTiles ? s : kDecMinTiles;
}

// The 8 x 8 matrix of 16-bit values held one row of pairs a lane group, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <typename T, int D, bool I8, int NRG>
__global__ void __launch_bounds__(32 * q8_decode_warps(NRG), 1)
q8_decode_kernel(const __grid_constant__ Q8Attend a, const __grid_constant__ Q8Tiles tl,
                 const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using P = DecodePlan<D, NRG>;
  constexpr int PQ = sizeof(T) == 4 ? 2 : 1;                                // fp16 planes of the queries
  constexpr int PP = std::is_same<T, __nv_bfloat16>::value ? 1 : 2;         // and of the weights
  constexpr int KS = D / 16;       // k-steps of the score MMA, and 32-bit words of a lane's key run
  constexpr int NO = D / 16;       // coordinate tiles of the output
  constexpr int VB = D / 8;        // bytes of a lane's value run, and its output coordinates
  constexpr int ROWS = 8 * NRG;
  constexpr int NS = P::NS;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + static_cast<size_t>(warp) * NS * P::STAGE;
  uint64_t* mbar = reinterpret_cast<uint64_t*>(smem + P::OFF_MBAR) + warp * NS;
  if (lane == 0)
    for (int s = 0; s < NS; ++s) tc::mbar_init(mbar + s, 1);
  __syncwarp();

  // shares are dealt across the blocks first, so that few of them still spread over every SM
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the merge may get ready; it waits for this grid's end
  const int workers = gridDim.x * P::WARPS;
  const int worker = blockIdx.x + gridDim.x * warp;
  Q8Flat flat;
  flat.load(a, tl, lane);
  const int64_t S = q8_share(flat.total, workers);
  const int64_t x0 = worker * S, x1 = min(x0 + S, flat.total);
  const bool wide = a.shift >= 5;  // a 32-token tile lies in one pool block
  uint32_t seq = 0;                // tiles consumed: stage seq % NS, phase parity (seq / NS) & 1
  bool failed = false;

  for (int64_t x = x0; x < x1;) {
    const Q8Place at = flat.at_tile(a, tl, lane, x);
    const int b = at.b;
    const int64_t seq0 = at.begin;
    const Q8Extent ext = at.ext;
    const Q8Span sp = at.sp;
    const int u = static_cast<int>(q8_div(x - seq0, ext.tiles));  // unit in the sequence: row tile, then KV head
    const int k0 = static_cast<int>(x - seq0 - static_cast<int64_t>(u) * ext.tiles);  // first key tile
    const int k1 = static_cast<int>(min(static_cast<int64_t>(ext.tiles), k0 + (x1 - x)));
    const int hk = u % a.Hkv, i0 = u / a.Hkv * tl.tpt;
    const int slot = x == x0 ? 0 : 1;
    const bool whole = k0 == 0 && k1 == ext.tiles;
    x += k1 - k0;
    const int nrow = min(tl.tpt, sp.count - i0) * a.G;
    const int t_end = sp.pos0 + i0 + nrow / a.G;                  // keys the row tile's last token sees
    const int end = min(min(k1 * kDecTile, a.T), t_end);
    const int ntiles = failed ? 0 : max(0, (end + kDecTile - 1) / kDecTile - k0);

    // lane l: the pool's scale blocks (16 rows each) of key tile k0 + 32 i + l, -1 past the end, and their scales
    auto blocks_of = [&](int i, int& r0, int& r1) {
      const int t0 = (k0 + 32 * i + lane) * kDecTile;
      r0 = r1 = -1;
      if (t0 < end) r0 = static_cast<int>(q8_row(a, b, hk, t0) >> 4);
      if (t0 + 16 < end) r1 = wide ? r0 + 1 : static_cast<int>(q8_row(a, b, hk, t0 + 16) >> 4);
    };
    auto scales_of = [&](int r0, int r1, float (&sc)[4]) {
      sc[0] = r0 >= 0 ? __ldg(a.kscales + r0) : 0.f;
      sc[1] = r1 >= 0 ? __ldg(a.kscales + r1) : 0.f;
      sc[2] = r0 >= 0 ? __ldg(a.vscales + r0) : 0.f;
      sc[3] = r1 >= 0 ? __ldg(a.vscales + r1) : 0.f;
    };
    int r0, r1, n0 = -1, n1 = -1;
    float sc[4], scn[4] = {0.f, 0.f, 0.f, 0.f};
    blocks_of(0, r0, r1);

    // tile i of the unit into stage (seq + i) % NS; rows past the end are other rows of the pool, masked below
    auto issue = [&](int i) {
      const int from = i & 31;
      const bool later = (i >> 5) != 0;  // relative to the batch the registers hold
      const int y0 = __shfl_sync(0xffffffffu, later ? n0 : r0, from), y1 = __shfl_sync(0xffffffffu, later ? n1 : r1, from);
      if (lane == 0) {
        const int s = static_cast<int>(seq % NS);
        uint8_t* st = ring + static_cast<size_t>(s) * P::STAGE;
        const bool two = !wide && y1 >= 0;
        mbar_arrive_expect_tx(mbar + s, static_cast<uint32_t>(2 * D * (wide ? 32 : two ? 32 : 16)));
        tma_load_2d(st, &kmap, 0, y0 * 16, mbar + s);
        tma_load_2d(st + P::PLANE, &vmap, 0, y0 * 16, mbar + s);
        if (two) {
          tma_load_2d(st + 16 * D, &kmap, 0, y1 * 16, mbar + s);
          tma_load_2d(st + P::PLANE + 16 * D, &vmap, 0, y1 * 16, mbar + s);
        }
      }
    };
    const uint32_t seq_unit = seq;
    for (int i = 0; i < NS && i < ntiles; ++i) {
      issue(i);
      ++seq;  // while issuing, seq names the stage
    }
    seq = seq_unit;
    scales_of(r0, r1, sc);

    // the query operand of this lane: row 8 n + g of group n, coordinates [D/4 t, D/4 t + D/4)
    uint32_t qf[NRG][PQ][KS][2];
    float f_row[NRG][2];
    int lim[NRG][2];               // rows 8 n + 2 t + {0, 1}, whose scores and output this lane holds: keys < lim are visible
#pragma unroll
    for (int n = 0; n < NRG; ++n) {
      const int r = 8 * n + g;
      const bool on = r < nrow;
      const int i = i0 + (on ? r / a.G : 0), h = hk * a.G + (on ? r % a.G : 0);
      const T* src =
          static_cast<const T*>(a.q) + (sp.first + i) * a.q_stride + static_cast<int64_t>(h) * D + (D / 4) * t;
      float v[KS][4], mx = 0.f;
#pragma unroll
      for (int s = 0; s < KS; s += 2) {
        Raw8<T> w;
        float y[8];
        if (on) w.load(src + 4 * s);
        else w.zero();
        w.values(y);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[s + (e >> 2)][e & 3] = y[e];
          mx = fmaxf(mx, fabsf(y[e]));
        }
      }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // a power of two that brings the row's largest magnitude to [2^13, 2^14): the planes keep their precision
      int ex = 0;
      if (mx > 0.f && isfinite(mx)) frexpf(mx, &ex);
      ex = max(-120, min(114, ex - 14));  // 114: the largest finite queries; -120: 2^-ex stays well inside fp32's range
      const float up = ldexpf(1.f, -ex), fr = a.mult * ldexpf(1.f, ex);
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if constexpr (PQ == 2) split_h2(v[s][2 * e] * up, v[s][2 * e + 1] * up, qf[n][0][s][e], qf[n][PQ - 1][s][e]);
          else qf[n][0][s][e] = pack_h2(v[s][2 * e] * up, v[s][2 * e + 1] * up);
        }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rr = 8 * n + 2 * t + e;
        f_row[n][e] = __shfl_sync(0xffffffffu, fr, 4 * (2 * t + e));
        lim[n][e] = rr < nrow ? min(sp.pos0 + i0 + rr / a.G + 1, end) : 0;
      }
    }

    float o[NRG][NO][4];           // coordinates VB g + 2 j + {0, 1} (registers 0 and 1, 2 and 3) of the two rows
    float m_run[NRG][2], l_part[NRG][2];
    float vref = 0.f;              // power of two the weights' value scales are relative to
#pragma unroll
    for (int n = 0; n < NRG; ++n) {
      m_run[n][0] = m_run[n][1] = -INFINITY;
      l_part[n][0] = l_part[n][1] = 0.f;
#pragma unroll
      for (int j = 0; j < NO; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][j][e] = 0.f;
    }

    for (int i = 0; i < ntiles; ++i) {
      const int bi = i & 31;
      if (bi == 0 && i > 0) {      // the next batch of 32 tiles moves in
        r0 = n0; r1 = n1;
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[e] = scn[e];
      }
      if (bi == 8 && i + 24 < ntiles) blocks_of((i >> 5) + 1, n0, n1);
      if (bi == 16 && i + 16 < ntiles) scales_of(n0, n1, scn);
      const float ks[2] = {__shfl_sync(0xffffffffu, sc[0], bi), __shfl_sync(0xffffffffu, sc[1], bi)};
      const float vs[2] = {__shfl_sync(0xffffffffu, sc[2], bi), __shfl_sync(0xffffffffu, sc[3], bi)};
      const int s = static_cast<int>(seq % NS);
      if (!__all_sync(0xffffffffu, tc::mbar_wait(mbar + s, (seq / NS) & 1))) {
        // a wait gave up: let this warp's copies in flight land, bounded again, before the block may exit
        failed = true;
        for (int j = 0; j < NS && i + j < ntiles; ++j) tc::mbar_wait(mbar + (seq + j) % NS, ((seq + j) / NS) & 1);
        break;
      }
      const uint8_t* sK = ring + static_cast<size_t>(s) * P::STAGE;
      const uint8_t* sV = sK + P::PLANE;
      const int t0 = (k0 + i) * kDecTile;
      const bool tail = t0 + kDecTile > sp.pos0 + i0 + 1 || t0 + kDecTile > end;  // some key is hidden from some row

      // S^T = K Q^T for 32 tokens: registers 0, 1 are token 16 h + g of rows 2 t, 2 t + 1, registers 2, 3 token + 8
      float sc4[NRG][2][4];
#pragma unroll
      for (int n = 0; n < NRG; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc4[n][h][e] = 0.f;
#pragma unroll
      for (int c = 0; c < KS / 4; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 x4 = *reinterpret_cast<const uint4*>(sK + q8_swz<D>(16 * h + g, (KS / 4) * t + c));
          const uint4 y4 = *reinterpret_cast<const uint4*>(sK + q8_swz<D>(16 * h + 8 + g, (KS / 4) * t + c));
          const uint32_t wx[4] = {x4.x, x4.y, x4.z, x4.w}, wy[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t a0, a1, a2, a3;
            q8_halves<I8>(wx[e], a0, a2);
            q8_halves<I8>(wy[e], a1, a3);
#pragma unroll
            for (int n = 0; n < NRG; ++n)
#pragma unroll
              for (int p = 0; p < PQ; ++p)
                mma16816(sc4[n][h], a0, a1, a2, a3, qf[n][p][4 * c + e][0], qf[n][p][4 * c + e][1]);
          }
        }

      const float vmax = fmaxf(vs[0], vs[1]);
      if (vmax > vref) {  // uniform
        // the power of two at or above vmax, from 2^-126 (subnormal scales) to 2^127: its reciprocal is exact
        const float up = __uint_as_float(min((__float_as_uint(vmax) + 0x7fffffu) & 0x7f800000u, 0x7f000000u));
        const float f = vref / up;
        vref = up;
#pragma unroll
        for (int n = 0; n < NRG; ++n)
#pragma unroll
          for (int j = 0; j < NO; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][j][e] *= f;
      }
      // weights are formed relative to vref and 2^14 up: at most 2^15 in fp16, the last plane's last step 2^-24
      // 1 / vref by its exponent (2^-127 is subnormal); vref = 0 where every scale so far, these two too, was 0
      const float vi = __uint_as_float(max(0x7f000000u - __float_as_uint(vref), 0x00400000u));
      const float vf[2] = {vs[0] * vi * 16384.f, vs[1] * vi * 16384.f};

      uint32_t pf[NRG][PP][2][2];
#pragma unroll
      for (int n = 0; n < NRG; ++n) {
        float p[2][4], mx[2] = {-INFINITY, -INFINITY}, m_use[2], alpha[2];  // [row][16 h + g, + 8]
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float f[2] = {f_row[n][r] * ks[0], f_row[n][r] * ks[1]};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int h = e >> 1;
            const float v = sc4[n][h][2 * (e & 1) + r] * f[h];
            p[r][e] = !tail || t0 + 16 * h + 8 * (e & 1) + g < lim[n][r] ? v : -INFINITY;
            mx[r] = fmaxf(mx[r], p[r][e]);
          }
        }
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
          mx[0] = fmaxf(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], x));
          mx[1] = fmaxf(mx[1], __shfl_xor_sync(0xffffffffu, mx[1], x));
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float m_new = fmaxf(m_run[n][r], mx[r]);
          m_use[r] = m_new == -INFINITY ? 0.f : m_new;
          alpha[r] = q8_ex2(m_run[n][r] - m_use[r]);
          m_run[n][r] = m_new;
          l_part[n][r] *= alpha[r];
        }
        if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
          for (int j = 0; j < NO; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][j][e] *= alpha[e & 1];
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[r][e] = q8_ex2(p[r][e] - m_use[r]);
            l_part[n][r] += p[r][e];
            p[r][e] *= vf[e >> 1];
          }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (PP == 2) {
            uint32_t hi, lo;
            split_h2(p[0][e], p[1][e], hi, lo);
            pf[n][0][e >> 1][e & 1] = transpose8x8(hi);
            pf[n][PP - 1][e >> 1][e & 1] = transpose8x8(lo);
          } else {
            pf[n][0][e >> 1][e & 1] = transpose8x8(pack_h2(p[0][e], p[1][e]));
          }
        }
      }

      // O^T += V^T P^T
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t vw[4][VB / 4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * h + 2 * t + (r & 1) + 8 * (r >> 1);
          if constexpr (VB == 16) {
            *reinterpret_cast<uint4*>(vw[r]) = *reinterpret_cast<const uint4*>(sV + q8_swz<D>(row, g));
          } else {
            *reinterpret_cast<uint2*>(vw[r]) =
                *reinterpret_cast<const uint2*>(sV + q8_swz<D>(row, g >> 1) + 8 * (g & 1));
          }
          if (tail && t0 + row >= end) {  // rows no query sees may hold anything (an e4m3 NaN): their weight is zero,
#pragma unroll
            for (int e = 0; e < VB / 4; ++e) vw[r][e] = 0u;  // so are they
          }
        }
#pragma unroll
        for (int e = 0; e < VB / 4; ++e) {
          uint32_t b0[4], b1[4];
          q8_pairs<I8>(vw[0][e], vw[1][e], b0);
          q8_pairs<I8>(vw[2][e], vw[3][e], b1);
#pragma unroll
          for (int n = 0; n < NRG; ++n)
#pragma unroll
            for (int p = 0; p < PP; ++p)
#pragma unroll
              for (int j = 0; j < 2; ++j)
                mma16816(o[n][2 * e + j], b0[2 * j], b0[2 * j + 1], b1[2 * j], b1[2 * j + 1], pf[n][p][h][0],
                         pf[n][p][h][1]);
        }
      }

      // the stage is free once every lane's reads of it are done
      fence_proxy_async();
      __syncwarp();
      if (i + NS < ntiles) issue(bi + NS);
      ++seq;
    }
    if (failed) {
      // what this warp owns from here on, this unit and the rest of its share, goes out as NaN
#pragma unroll
      for (int n = 0; n < NRG; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) m_run[n][r] = l_part[n][r] = __int_as_float(0x7fc00000);
    }

    // the rows' outputs, or their partials when the unit is cut
    const float unscale = 1.f / 16384.f;  // vref comes last: with it, the factor could leave fp32's normal range
#pragma unroll
    for (int n = 0; n < NRG; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float l = l_part[n][r];
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
        const int row = 8 * n + 2 * t + r;
        if (row >= nrow) continue;
        const float f = !whole ? unscale : l == 0.f ? 0.f : unscale / l;  // NaN stays
        float y[VB];
#pragma unroll
        for (int j = 0; j < NO; ++j) {
          y[2 * j] = whole && l == 0.f ? 0.f : o[n][j][r] * f * vref;
          y[2 * j + 1] = whole && l == 0.f ? 0.f : o[n][j][2 + r] * f * vref;
        }
        if (whole) {
          const int64_t orow = (sp.first + i0 + row / a.G) * a.Hq + static_cast<int64_t>(hk) * a.G + row % a.G;
          T* dst = static_cast<T*>(a.out) + orow * D + VB * g;
#pragma unroll
          for (int j = 0; j < VB; j += 8) store8(dst + j, *reinterpret_cast<float(*)[8]>(y + j));
        } else {
          const int64_t part = (static_cast<int64_t>(worker) * 2 + slot) * ROWS + row;
          float* dst = a.ws_o + part * D + VB * g;
#pragma unroll
          for (int j = 0; j < VB; j += 8) store8(dst + j, *reinterpret_cast<float(*)[8]>(y + j));
          if (g == 0) {
            a.ws_m[part] = m_run[n][r];
            a.ws_l[part] = l;
          }
        }
      }
  }
  if (failed && lane == 0) atomicOr(a.status, 1u);
}

// Merge of the units cut by a share's edge (q8_merge_row).  Rows that a worker finished are left alone; rows of sequences
// without keys get zeros.  Launched as a programmatic dependent of the decode kernel.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kMergeWarps)
q8_decode_merge_kernel(const __grid_constant__ Q8Attend a, const __grid_constant__ Q8Tiles tl, int rows, int workers) {
  const int lane = threadIdx.x & 31;
  const int per = tl.tpt * a.G, r = static_cast<int>(blockIdx.x) % per, unit = static_cast<int>(blockIdx.x) / per;
  const int hk = unit % a.Hkv;
  int b;
  int64_t i0;
  q8_tile(a, tl, unit / a.Hkv, lane, b, i0);
  int64_t total;
  const Q8Place at = q8_place(a, tl, lane, b, total);
  const Q8Span sp = at.sp;
  // every block waits, those without a row too: this grid's end stands for the attention kernel's
  const auto wait = [] { asm volatile("griddepcontrol.wait;\n" ::: "memory"); };
  if (!q8_tile_live(a, tl, sp, i0, threadIdx.x)) return wait();
  if (r >= min(tl.tpt, sp.count - static_cast<int>(i0)) * a.G) return wait();
  const int64_t S = q8_share(total, workers);
  const Q8Extent ext = at.ext;
  const int64_t p0 = at.begin + (q8_div(i0, tl.tpt) * a.Hkv + hk) * ext.tiles, p1 = p0 + ext.tiles;  // the unit's flat tiles
  const int w0 = static_cast<int>(q8_div(p0, S)), n = p1 > p0 ? static_cast<int>(q8_div(p1 - 1, S)) - w0 + 1 : 0;
  wait();                                                 // the partials are complete and visible after this
  if (n == 1) return;                                     // one worker finished it
  // partial k of the unit: slot 0 of worker w0 + k, but slot 1 of w0 where the unit begins inside its share
  const int64_t first = (static_cast<int64_t>(w0) * 2 + (p0 > w0 * S ? 1 : 0)) * rows + r;
  const int64_t rest = static_cast<int64_t>(w0) * 2 * rows + r;
  const int64_t orow = (sp.first + i0 + r / a.G) * a.Hq + static_cast<int64_t>(hk) * a.G + r % a.G;
  q8_merge_row<T, D, kMergeWarps>(a, n, [&](int k) { return k == 0 ? first : rest + static_cast<int64_t>(k) * 2 * rows; }, orow);
}

}  // namespace axr
