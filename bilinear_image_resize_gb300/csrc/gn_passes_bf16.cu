// The pass kernels of group norm (gn_passes.h) for bfloat16 maps.
#include <algorithm>

#include "gn_passes.h"

namespace rz {
template cudaError_t gn_passes_forward<__nv_bfloat16>(const GnArgs &, int, bool, void *);
template cudaError_t gn_passes_backward<__nv_bfloat16>(const GnArgs &, int, bool, void *);
}  // namespace rz
