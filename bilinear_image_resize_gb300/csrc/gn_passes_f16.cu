// The pass kernels of group norm (gn_passes.h) for float16 maps.
#include <algorithm>

#include "gn_passes.h"

namespace rz {
template cudaError_t gn_passes_forward<__half>(const GnArgs &, int, bool, void *);
template cudaError_t gn_passes_backward<__half>(const GnArgs &, int, bool, void *);
}  // namespace rz
