// The product's kernels with scales of 128 for A E5M2, W E5M2.
#include "block_impl.h"

namespace mxg {
template hipError_t launch_block_fmt<kE5M2, kE5M2>(int, bool, const BlockLinArgs&, hipStream_t);
}
