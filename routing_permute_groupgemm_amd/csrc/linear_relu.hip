#include "linear_tiles.hpp"

namespace moe {

int launch_linear_relu(const GemmParams& p, int tiles, hipStream_t s) { return launch_linear_act<MOE_ACT_RELU>(p, tiles, s); }

}  // namespace moe
