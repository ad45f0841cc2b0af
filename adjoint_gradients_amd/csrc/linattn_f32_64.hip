// linattn_f32_64.hip -- the linear-attention kernels of io type f32 for q and k
// heads padded to 64 channels.
#include "linattn.inl"

namespace la {

hipError_t launch_f32_64(Kernel k, int dv, const Args& a, hipStream_t st) {
  if (padded(dv) == 64) return launch_kind<float, 64, 64>(k, a, st);
  return launch_kind<float, 64, 128>(k, a, st);
}

}  // namespace la
