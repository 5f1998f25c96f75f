// Attention over the paged cache: the kernels for MXFP8, results in fp32 with more than 16 rows a key head.
#include "attend_kernel.h"

int launch_attend_mxfp8_fp32(const AttendArgs& a, const AttendPlan& p, uint8_t* ws, hipStream_t stream) {
  return launch_format<MXFP4_FMT_MXFP8, true>(a, p, ws, stream);
}
