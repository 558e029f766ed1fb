// svt_gated_f32.hip - products with a gate and their gradients for float32 rows
#define SVT_GATED_INSTANTIATE
#include "svt_gated.h"

namespace svt {
template int gated_forward<float>(const char *, GatedArgs, const GatedPlan &, void *);
template int gated_backward<float>(const char *, GatedArgs, const GatedPlan &, void *);
}  // namespace svt
