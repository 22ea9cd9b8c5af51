// Layer norm of fp32 rows that stay on chip.
#include "train_norm_rows.h"

namespace traingb {

const NormKernels& norm_kernels_fp32(int y_type) {
  static constexpr NormKernels kernels[3] = {norm_kernels<TRAIN_FP32, TRAIN_BF16>(),
                                             norm_kernels<TRAIN_FP32, TRAIN_FP16>(),
                                             norm_kernels<TRAIN_FP32, TRAIN_FP32>()};
  return kernels[y_type];
}

}  // namespace traingb
