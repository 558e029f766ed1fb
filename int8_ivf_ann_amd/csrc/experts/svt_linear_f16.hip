// svt_linear_f16.hip - products of float16 rows with 4-bit weights

#include "svt_linear.h"

namespace svt {

template int linear_rows<f16>(const char *, LinearArgs, int32_t, void *);

}  // namespace svt
