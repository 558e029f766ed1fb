// svt_linear_f32.hip - products of float32 rows with 4-bit weights

#include "svt_linear.h"

namespace svt {

template int linear_rows<float>(const char *, LinearArgs, int32_t, void *);

}  // namespace svt
