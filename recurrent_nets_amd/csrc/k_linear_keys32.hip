// Linear attention in chunks (linear.h) for keys of up to 32 columns.
#include "linear.h"

namespace slstm {

hipError_t launch_linear_keys32(bool bf16, int value_blocks, const LinLaunch& a, LinPass pass, hipStream_t st) {
  return lin_launch_keys<1>(bf16, value_blocks, a, pass, st);
}

}  // namespace slstm
