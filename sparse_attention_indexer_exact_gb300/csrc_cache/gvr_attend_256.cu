// gvr_attend_256.cu -- the attention kernels for head_dim 256.
#include "gvr_attend.cuh"

namespace gvrc {

KernelInfo attend_256() { return info<256, 1>(); }

}  // namespace gvrc
