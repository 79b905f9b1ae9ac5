// gvr_shared_128.cu -- the kernels of attend_shared for head_dim 128.
#include "gvr_shared.cuh"

namespace gvrc {

SharedInfo shared_128() { return shared_info<128>(); }

}  // namespace gvrc
