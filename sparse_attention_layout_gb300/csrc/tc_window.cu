// Tensor-core paths of the windowed attention: none yet, every call takes the
// CUDA-core kernels.
#include "window.h"

namespace bsp {
namespace win {

int launch_forward_tc(Call&) { return BSP_ERR_UNSUPPORTED; }
int launch_backward_tc(Call&) { return BSP_ERR_UNSUPPORTED; }

}  // namespace win
}  // namespace bsp
