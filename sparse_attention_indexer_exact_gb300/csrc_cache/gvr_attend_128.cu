// gvr_attend_128.cu -- the attention kernels for head_dim 128.
#include "gvr_attend.cuh"

namespace gvrc {

KernelInfo attend_128(int i) { return i == 0 ? info<128, 1>() : info<128, 2>(); }

}  // namespace gvrc
