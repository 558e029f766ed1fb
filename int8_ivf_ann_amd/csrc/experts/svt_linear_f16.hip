// svt_linear_f16.hip - products of float16 rows with 4-bit weights

#include "svt_linear.h"

namespace svt {

template void linear_rows<f16>(LinearArgs, int32_t, hipStream_t);

}  // namespace svt
