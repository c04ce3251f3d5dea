// Tiled products of the linear and gated calls on bf16 operands.
#include "linear_launch_tile.h"

namespace convfwd {

template hipError_t launch_product<__bf16>(const ProductArgs&, int, int, bool, bool, hipStream_t);
template hipError_t launch_pair<__bf16>(const PairArgs&, int, bool, hipStream_t);

}  // namespace convfwd
