// svt_linear_bf16.hip - products of bfloat16 rows with 4-bit weights

#include "svt_linear.h"

namespace svt {

template void linear_rows<bf16>(LinearArgs, int32_t, hipStream_t);

}  // namespace svt
