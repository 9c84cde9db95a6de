// cp_linear_dx.hip - cp_linear_dx's product: dx[m][k] from rows of dz and the
// columns of w.
#include "cp_linear_tile.h"

namespace cpk {

hipError_t linear_rows_by_columns(const LinearArgs &a)
{
    if (a.dtype == kBF16) return launch_linear<kBF16, false, true, kBF16>(a);
    if (a.dtype == kF16) return launch_linear<kF16, false, true, kF16>(a);
    return launch_linear<kF32, false, true, kF32>(a);
}

}  // namespace cpk
