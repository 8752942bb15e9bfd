#include "linear_tiles.hpp"

namespace moe {

int launch_linear_gelu(const GemmParams& p, int tiles, hipStream_t s) { return launch_linear_act<MOE_ACT_GELU>(p, tiles, s); }

}  // namespace moe
