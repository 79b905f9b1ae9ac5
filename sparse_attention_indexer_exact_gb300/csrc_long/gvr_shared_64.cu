// gvr_shared_64.cu -- the kernels of attend_shared for head_dim 64.
#include "gvr_shared.cuh"

namespace gvrc {

SharedInfo shared_64() { return shared_info<64>(); }

}  // namespace gvrc
