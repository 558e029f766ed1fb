// svt_gated_f16.hip - products with a gate and their gradients for float16 rows
#define SVT_GATED_INSTANTIATE
#include "svt_gated.h"

namespace svt {
template int gated_forward<f16>(const char *, GatedArgs, const GatedPlan &, void *);
template int gated_backward<f16>(const char *, GatedArgs, const GatedPlan &, void *);
}  // namespace svt
