// tk_rows_f16_r32.hip -- the row operators' kernels for binary16 with a float residual stream.
#include "tk_rows.h"

namespace tk {
RowTable rows_f16_r32() { return RowKernels<f16_t, float>::table(); }
}  // namespace tk
