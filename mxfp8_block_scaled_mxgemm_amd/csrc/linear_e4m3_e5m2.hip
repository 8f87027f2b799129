// The product's kernels for A E4M3, W E5M2.
#include "linear_impl.h"

namespace mxg {
template hipError_t launch_linear_fmt<kE4M3, kE5M2>(int, bool, const LinArgs&, hipStream_t);
}
