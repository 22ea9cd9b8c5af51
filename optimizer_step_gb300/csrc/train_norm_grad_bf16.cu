// Layer norm's backward pass for bf16 rows that stay on chip.
#include "train_norm_grad_rows.h"

namespace traingb {

const NormGradKernels& norm_grad_kernels_bf16(int y_type) {
  static constexpr NormGradKernels kernels[3] = {norm_grad_kernels<TRAIN_BF16, TRAIN_BF16>(),
                                                 norm_grad_kernels<TRAIN_BF16, TRAIN_FP16>(),
                                                 norm_grad_kernels<TRAIN_BF16, TRAIN_FP32>()};
  return kernels[y_type];
}

}  // namespace traingb
