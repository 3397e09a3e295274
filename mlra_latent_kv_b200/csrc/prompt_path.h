// Which kernel a prompt takes: a rule on the host alone, before anything is
// enqueued.
#pragma once

#include "../../include/mlra.h"

namespace mlra {

enum class PromptPath { kTc, kSimt, kNoShape, kNoRegisters };

// fits: the tcgen05 kernel takes the dims and the layout.  regs: the registers
// of a thread that the compiler gave it, want: those that its warp roles share
// out anew.  Compiled otherwise it could not run, and the CUDA-core kernel does
// the work unless the caller insists.
inline PromptPath prompt_path(mlra_kernel kernel, bool fits, int regs, int want) {
  if (kernel == MLRA_KERNEL_SIMT) return PromptPath::kSimt;
  if (fits && regs == want) return PromptPath::kTc;
  if (kernel != MLRA_KERNEL_TC) return PromptPath::kSimt;
  return fits ? PromptPath::kNoRegisters : PromptPath::kNoShape;
}

}  // namespace mlra
