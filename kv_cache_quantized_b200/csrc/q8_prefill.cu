// Launcher of the tcgen05 attention over the 8-bit cache (q8_prefill.cuh).
#include "launch.h"
#include "q8_merge.cuh"
#include "q8_prefill.cuh"

namespace axr {
namespace {

template <typename T, int D, bool I8>
axr_status launch(const Q8Attend& a, const Q8Tiles& tl, cudaStream_t st, const char* w) {
  auto k = q8_prefill_kernel<T, D, I8>;
  const axr_status rs = ensure_smem(k, PrefillPlan<D>::bytes, w);
  if (rs != AXR_OK) return rs;
  k<<<static_cast<unsigned>(tl.tiles * a.Hkv * a.splits), kPfThreads, PrefillPlan<D>::bytes, st>>>(a, tl);
  if (a.splits > 1) {
    auto merge = a.splits <= 8 ? q8_merge_kernel<T, D, 1> : q8_merge_kernel<T, D, kMergeWarps>;
    // the merge keeps the attention kernel's split of L1: another one would have to wait for every SM to drain
    cudaFuncSetAttribute(merge, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    // a warp a row until the warps fill the SMs, then up to 8 rows each: many tiles have no work
    const int64_t units = tl.tiles * a.Hkv, warps = units * a.rows, resident = 64 * kSmCount;
    const int each = static_cast<int>(warps <= resident ? 1 : warps < 8 * resident ? (warps + resident - 1) / resident : 8);
    const int per = a.splits <= 8 ? kMergeWarps * each : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(units * ((a.rows + per - 1) / per)));
    cfg.blockDim = dim3(32 * kMergeWarps);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, merge, a, tl, a.rows, each);
  }
  return check_launch(w);
}

template <typename T>
axr_status by_d(int d, bool i8, const Q8Attend& a, const Q8Tiles& tl, cudaStream_t st, const char* w) {
  if (d == 64) return i8 ? launch<T, 64, true>(a, tl, st, w) : launch<T, 64, false>(a, tl, st, w);
  return i8 ? launch<T, 128, true>(a, tl, st, w) : launch<T, 128, false>(a, tl, st, w);
}

}  // namespace

axr_status q8_prefill_launch(bool half, int d, bool i8, const Q8Attend& a, const Q8Tiles& tl, cudaStream_t st,
                             const char* w) {
  return half ? by_d<__half>(d, i8, a, tl, st, w) : by_d<__nv_bfloat16>(d, i8, a, tl, st, w);
}

}  // namespace axr
