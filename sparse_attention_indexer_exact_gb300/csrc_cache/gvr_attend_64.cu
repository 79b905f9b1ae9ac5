// gvr_attend_64.cu -- the attention kernels for head_dim 64.
#include "gvr_attend.cuh"

namespace gvrc {

KernelInfo attend_64(int i) { return i == 0 ? info<64, 1>() : i == 1 ? info<64, 2>() : info<64, 4>(); }

}  // namespace gvrc
