// tk_rows_f32.hip -- the row operators' kernels for float.
#include "tk_rows.h"

namespace tk {
RowTable rows_f32() { return RowKernels<float, float>::table(); }
}  // namespace tk
