// The distillation loss of bf16 logits in rows that stay in shared memory or pass through it.
#include "train_distill_rows.h"

namespace traingb {

const DistillKernels& distill_kernels_bf16() {
  static constexpr DistillKernels kernels = distill_kernels<TRAIN_BF16>();
  return kernels;
}

}  // namespace traingb
