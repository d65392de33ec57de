#include "rope_norm_kernel.cuh"

namespace block_ops {
template RopeKernel pick_rope<true>(int, int, bool, bool);
}
