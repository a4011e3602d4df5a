// w4_kernel for one of its three uses; a translation unit each, so that they
// compile side by side.
#include "w4_kernel.cuh"

namespace moe {
namespace w4 {

cudaError_t launch_fc1(int group, int K, bool wide, const Args& a, cudaStream_t s) {
  return launch_mode<FC1>(group, K, wide, a, s);
}

}  // namespace w4
}  // namespace moe
