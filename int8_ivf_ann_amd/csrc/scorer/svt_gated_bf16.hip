// svt_gated_bf16.hip - products with a gate and their gradients for bfloat16 rows
#define SVT_GATED_INSTANTIATE
#include "svt_gated.h"

namespace svt {
template int gated_forward<bf16>(const char *, GatedArgs, const GatedPlan &, void *);
template int gated_backward<bf16>(const char *, GatedArgs, const GatedPlan &, void *);
}  // namespace svt
