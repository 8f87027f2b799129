// The product's kernels with scales of 128 for A E4M3, W E4M3.
#include "block_impl.h"

namespace mxg {
template hipError_t launch_block_fmt<kE4M3, kE4M3>(int, bool, const BlockLinArgs&, hipStream_t);
}
