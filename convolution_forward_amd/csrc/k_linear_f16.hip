// Tiled products of the linear and gated calls on f16 operands.
#include "linear_launch_tile.h"

namespace convfwd {

template hipError_t launch_product<_Float16>(const ProductArgs&, int, int, bool, bool, hipStream_t);
template hipError_t launch_pair<_Float16>(const PairArgs&, int, bool, hipStream_t);

}  // namespace convfwd
