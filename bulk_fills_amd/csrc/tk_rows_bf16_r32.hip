// tk_rows_bf16_r32.hip -- the row operators' kernels for bfloat16 with a float residual stream.
#include "tk_rows.h"

namespace tk {
RowTable rows_bf16_r32() { return RowKernels<bf16_t, float>::table(); }
}  // namespace tk
