// Attention over the paged cache: the kernels for MXFP4, results in fp32 with more than 16 rows a key head.
#include "attend_kernel.h"

int launch_attend_mxfp4_fp32(const AttendArgs& a, const AttendPlan& p, uint8_t* ws, hipStream_t stream) {
  return launch_format<MXFP4_FMT_MXFP4, true>(a, p, ws, stream);
}
