// svt_linear_f32.hip - products of float32 rows with 4-bit weights

#include "svt_linear.h"

namespace svt {

template void linear_rows<float>(LinearArgs, int32_t, hipStream_t);

}  // namespace svt
