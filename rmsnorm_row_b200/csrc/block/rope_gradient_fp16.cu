#include "rope_norm_kernel.cuh"

namespace block_ops {
template RopeKernel pick_rope_gradient<true>(int, int, bool, bool, bool);
}
