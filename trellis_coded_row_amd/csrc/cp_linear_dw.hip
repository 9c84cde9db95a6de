// cp_linear_dw.hip - cp_linear_dw's product: dw[n][k] from the columns of dz
// and of x, in 32 bits.
#include "cp_linear_tile.h"

namespace cpk {

hipError_t linear_columns_by_columns(const LinearArgs &a)
{
    if (a.dtype == kBF16) return launch_linear<kBF16, true, true, kF32>(a);
    if (a.dtype == kF16) return launch_linear<kF16, true, true, kF32>(a);
    return launch_linear<kF32, true, true, kF32>(a);
}

}  // namespace cpk
