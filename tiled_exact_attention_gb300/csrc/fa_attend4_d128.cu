// fa_fwd_kvcache_int4 for head dimension 128 (a translation unit of its own for the build's sake).
#include "fa_attend4.cuh"

namespace fa {

cudaError_t attend4_d128(const Attend4Params& p, int dtype, int sms, Attend4Plan* plan, cudaStream_t stream) {
  if (p.group == 128) return attend4::launch_rows<128, 1>(p, dtype, sms, plan, stream);
  if (p.group == 64) return attend4::launch_rows<128, 2>(p, dtype, sms, plan, stream);
  if (p.group == 32) return attend4::launch_rows<128, 4>(p, dtype, sms, plan, stream);
  return cudaErrorInvalidValue;
}

}  // namespace fa
