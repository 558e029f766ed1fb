// svt_linear_bf16.hip - products of bfloat16 rows with 4-bit weights

#include "svt_linear.h"

namespace svt {

template int linear_rows<bf16>(const char *, LinearArgs, int32_t, void *);

}  // namespace svt
