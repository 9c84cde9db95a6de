// cp_linear.hip - cp_linear's product: y[m][n] from rows of x and rows of w.
#include "cp_linear_tile.h"

namespace cpk {

uint64_t linear_workspace_bytes(uint64_t m, uint64_t n, uint64_t k, int dtype)
{
    const uint64_t a = workspace_of(cut_of(m, n, k, dtype, true), m, n), b = workspace_of(cut_of(m, n, k, dtype, false), m, n);
    return a > b ? a : b;
}

hipError_t linear_rows_by_rows(const LinearArgs &a)
{
    if (a.dtype == kBF16) return launch_linear<kBF16, false, false, kBF16>(a);
    if (a.dtype == kF16) return launch_linear<kF16, false, false, kF16>(a);
    return launch_linear<kF32, false, false, kF32>(a);
}

}  // namespace cpk
