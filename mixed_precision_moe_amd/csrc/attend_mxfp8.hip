// Attention over the paged cache: the kernels for MXFP8.
#include "attend_kernel.h"

int launch_attend_mxfp8(const AttendArgs& a, const AttendPlan& p, uint8_t* ws, hipStream_t stream) {
  return launch_format<MXFP4_FMT_MXFP8>(a, p, ws, stream);
}
