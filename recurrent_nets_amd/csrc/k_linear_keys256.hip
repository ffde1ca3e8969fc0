// Linear attention in chunks (linear.h) for keys of 129 to 256 columns.
#include "linear.h"

namespace slstm {

hipError_t launch_linear_keys256(bool bf16, int value_blocks, const LinLaunch& a, LinPass pass, hipStream_t st) {
  return lin_launch_keys<8>(bf16, value_blocks, a, pass, st);
}

}  // namespace slstm
