// Linear attention in chunks (linear.h) for keys of 33 to 64 columns.
#include "linear.h"

namespace slstm {

hipError_t launch_linear_keys64(bool bf16, int value_blocks, const LinLaunch& a, LinPass pass, hipStream_t st) {
  return lin_launch_keys<2>(bf16, value_blocks, a, pass, st);
}

}  // namespace slstm
