// Attention over the paged cache: the kernels for MXFP4.
#include "attend_kernel.h"

int launch_attend_mxfp4(const AttendArgs& a, const AttendPlan& p, uint8_t* ws, hipStream_t stream) {
  return launch_format<MXFP4_FMT_MXFP4>(a, p, ws, stream);
}
