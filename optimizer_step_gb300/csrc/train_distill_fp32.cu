// The distillation loss of fp32 logits in rows that stay in shared memory or pass through it.
#include "train_distill_rows.h"

namespace traingb {

const DistillKernels& distill_kernels_fp32() {
  static constexpr DistillKernels kernels = distill_kernels<TRAIN_FP32>();
  return kernels;
}

}  // namespace traingb
