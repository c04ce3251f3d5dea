// Tiled products of the linear and gated calls on f32 operands.
#include "linear_launch_tile.h"

namespace convfwd {

template hipError_t launch_product<float>(const ProductArgs&, int, int, bool, bool, hipStream_t);
template hipError_t launch_pair<float>(const PairArgs&, int, bool, hipStream_t);

}  // namespace convfwd
