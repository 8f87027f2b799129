// The product's kernels with scales of 128 for A E5M2, W E4M3.
#include "block_impl.h"

namespace mxg {
template hipError_t launch_block_fmt<kE5M2, kE4M3>(int, bool, const BlockLinArgs&, hipStream_t);
}
