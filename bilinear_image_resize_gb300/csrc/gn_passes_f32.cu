// The pass kernels of group norm (gn_passes.h) for float32 maps.
#include <algorithm>

#include "gn_passes.h"

namespace rz {
template cudaError_t gn_passes_forward<float>(const GnArgs &, int, bool, void *);
template cudaError_t gn_passes_backward<float>(const GnArgs &, int, bool, void *);
}  // namespace rz
