// gvr_shared_256.cu -- the kernels of attend_shared for head_dim 256.
#include "gvr_shared.cuh"

namespace gvrc {

SharedInfo shared_256() { return shared_info<256>(); }

}  // namespace gvrc
