// The linear layers' kernels for bf16 operands.
#include "linear_kernels.cuh"

namespace ep {
namespace linear {

Kernel bf16_kernel(bool pair, bool split, int bn, bool parts) {
    if (pair) return parts ? linear_pair_kernel<false, true> : linear_pair_kernel<false, false>;
    if (split)
        return bn == 32 ? linear_kernel<false, true, 32> : bn == 64 ? linear_kernel<false, true, 64> : linear_kernel<false, true, 128>;
    return bn == 32 ? linear_kernel<false, false, 32> : bn == 64 ? linear_kernel<false, false, 64> : linear_kernel<false, false, 128>;
}

}  // namespace linear
}  // namespace ep
