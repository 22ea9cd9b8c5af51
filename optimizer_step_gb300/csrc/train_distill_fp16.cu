// The distillation loss of fp16 logits in rows that stay in shared memory or pass through it.
#include "train_distill_rows.h"

namespace traingb {

const DistillKernels& distill_kernels_fp16() {
  static constexpr DistillKernels kernels = distill_kernels<TRAIN_FP16>();
  return kernels;
}

}  // namespace traingb
