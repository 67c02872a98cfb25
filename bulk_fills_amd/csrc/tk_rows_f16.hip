// tk_rows_f16.hip -- the row operators' kernels for binary16, with a residual stream of the
// same type.
#include "tk_rows.h"

namespace tk {
RowTable rows_f16() { return RowKernels<f16_t, f16_t>::table(); }
}  // namespace tk
