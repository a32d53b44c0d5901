// y[r] = x[r] W_e(r)^T in 16 bits: the tile kernel's first pass.
#include "rows_tile.h"

namespace mxmoe {
namespace rows {

hipError_t launch_forward(const RowsArgs& a, const RowsChoice& c, RowType in, RowType out, hipStream_t st) {
  return launch_pass<Pass::kForward>(a, c, in, out, st);
}

}  // namespace rows
}  // namespace mxmoe
