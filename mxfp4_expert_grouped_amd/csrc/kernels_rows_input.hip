// dx[r] = dy[r] W_e(r) in 16 bits: the gradient of the rows.
#include "rows_tile.h"

namespace mxmoe {
namespace rows {

hipError_t launch_input(const RowsArgs& a, const RowsChoice& c, RowType in, RowType out, hipStream_t st) {
  return launch_pass<Pass::kInput>(a, c, in, out, st);
}

}  // namespace rows
}  // namespace mxmoe
