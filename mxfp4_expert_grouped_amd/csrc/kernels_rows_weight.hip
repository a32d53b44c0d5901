// dW_e = the sum over its rows of dy[r]^T x[r] in 16 bits: the gradient of the weights.
#include "rows_tile.h"

namespace mxmoe {
namespace rows {

hipError_t launch_weight(const RowsArgs& a, const RowsChoice& c, RowType in, RowType out, hipStream_t st) {
  return launch_pass<Pass::kWeight>(a, c, in, out, st);
}

}  // namespace rows
}  // namespace mxmoe
