// linattn_bf16_64.hip -- the linear-attention kernels of io type bf16 for q and k
// heads padded to 64 channels.
#include "linattn.inl"

namespace la {

hipError_t launch_bf16_64(Kernel k, int dv, const Args& a, hipStream_t st) {
  if (padded(dv) == 64) return launch_kind<ssm::bf16_t, 64, 64>(k, a, st);
  return launch_kind<ssm::bf16_t, 64, 128>(k, a, st);
}

}  // namespace la
