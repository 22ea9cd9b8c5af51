// Layer norm of bf16 rows that stay on chip.
#include "train_norm_rows.h"

namespace traingb {

const NormKernels& norm_kernels_bf16(int y_type) {
  static constexpr NormKernels kernels[3] = {norm_kernels<TRAIN_BF16, TRAIN_BF16>(),
                                             norm_kernels<TRAIN_BF16, TRAIN_FP16>(),
                                             norm_kernels<TRAIN_BF16, TRAIN_FP32>()};
  return kernels[y_type];
}

}  // namespace traingb
