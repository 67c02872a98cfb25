// tk_rows_bf16.hip -- the row operators' kernels for bfloat16, with a residual stream of the
// same type.
#include "tk_rows.h"

namespace tk {
RowTable rows_bf16() { return RowKernels<bf16_t, bf16_t>::table(); }
}  // namespace tk
