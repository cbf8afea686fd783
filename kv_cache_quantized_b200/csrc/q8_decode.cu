// Launcher of the decode kernel over the 8-bit cache (q8_decode.cuh) and its merge.
#include "launch.h"
#include "q8_decode.cuh"

namespace axr {
namespace {

template <typename T, int D, bool I8, int NRG>
axr_status launch(int grid, const Q8Attend& a, const Q8Tiles& tl, cudaStream_t st, const char* w) {
  using P = DecodePlan<D, NRG>;
  auto k = q8_decode_kernel<T, D, I8, NRG>;
  axr_status rs = ensure_smem(k, P::bytes, w);
  if (rs != AXR_OK) return rs;
  const size_t rows = (static_cast<size_t>(a.num_blocks) * a.Hkv) << a.shift;
  if (rows + kDecTile >= (static_cast<size_t>(1) << 31))
    return set_error(AXR_EUNSUPPORTED, "%s: %zu pool rows exceed the 2^31 a TMA coordinate addresses", w, rows);
  const int box = a.shift >= 5 ? 32 : 16;
  CUtensorMap kmap, vmap;
  if ((rs = encode_byte_map(&kmap, a.kcodes, rows, D, box, w)) != AXR_OK) return rs;
  if ((rs = encode_byte_map(&vmap, a.vcodes, rows, D, box, w)) != AXR_OK) return rs;
  k<<<static_cast<unsigned>(grid), 32 * P::WARPS, P::bytes, st>>>(a, tl, kmap, vmap);
  // the merge keeps the decode kernel's split of L1: another one would have to wait for every SM to drain
  cudaFuncSetAttribute(q8_decode_merge_kernel<T, D>, cudaFuncAttributePreferredSharedMemoryCarveout,
                       cudaSharedmemCarveoutMaxShared);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tl.tiles * a.Hkv * tl.tpt * a.G));
  cfg.blockDim = dim3(32 * kMergeWarps);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaLaunchKernelEx(&cfg, q8_decode_merge_kernel<T, D>, a, tl, 8 * NRG, grid * P::WARPS);
  return check_launch(w);
}

template <typename T, int D>
axr_status by_kind(bool i8, int nrg, int grid, const Q8Attend& a, const Q8Tiles& tl, cudaStream_t st, const char* w) {
  if (i8) return nrg == 1 ? launch<T, D, true, 1>(grid, a, tl, st, w) : launch<T, D, true, 2>(grid, a, tl, st, w);
  return nrg == 1 ? launch<T, D, false, 1>(grid, a, tl, st, w) : launch<T, D, false, 2>(grid, a, tl, st, w);
}

template <typename T>
axr_status by_d(int d, bool i8, int nrg, int grid, const Q8Attend& a, const Q8Tiles& tl, cudaStream_t st,
                const char* w) {
  return d == 64 ? by_kind<T, 64>(i8, nrg, grid, a, tl, st, w) : by_kind<T, 128>(i8, nrg, grid, a, tl, st, w);
}

}  // namespace

axr_status q8_decode_launch(axr_dtype dtype, int d, bool i8, int nrg, int grid, const Q8Attend& a, const Q8Tiles& tl,
                            cudaStream_t st, const char* w) {
  if (dtype == AXR_F16) return by_d<__half>(d, i8, nrg, grid, a, tl, st, w);
  if (dtype == AXR_BF16) return by_d<__nv_bfloat16>(d, i8, nrg, grid, a, tl, st, w);
  return by_d<float>(d, i8, nrg, grid, a, tl, st, w);
}

}  // namespace axr
