// Linear attention in chunks (linear.h) for keys of 65 to 128 columns.
#include "linear.h"

namespace slstm {

hipError_t launch_linear_keys128(bool bf16, int value_blocks, const LinLaunch& a, LinPass pass, hipStream_t st) {
  return lin_launch_keys<4>(bf16, value_blocks, a, pass, st);
}

}  // namespace slstm
