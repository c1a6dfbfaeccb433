// The linear layers' kernels for e4m3 operands.
#include "linear_kernels.cuh"

namespace ep {
namespace linear {

Kernel e4m3_kernel(bool pair, bool split, int bn) {
    if (pair) return linear_pair_kernel<true, true>;
    if (split)
        return bn == 32 ? linear_kernel<true, true, 32> : bn == 64 ? linear_kernel<true, true, 64> : linear_kernel<true, true, 128>;
    return bn == 32 ? linear_kernel<true, false, 32> : bn == 64 ? linear_kernel<true, false, 64> : linear_kernel<true, false, 128>;
}

}  // namespace linear
}  // namespace ep
