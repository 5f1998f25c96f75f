// Attention over the paged cache: the kernels for MXFP8, results in bf16, and all with up to 16 rows a key head.
#include "attend_kernel.h"

int launch_attend_mxfp8(const AttendArgs& a, const AttendPlan& p, uint8_t* ws, hipStream_t stream) {
  if (a.out_fp32 && p.nt > 1) return launch_attend_mxfp8_fp32(a, p, ws, stream);
  return launch_format<MXFP4_FMT_MXFP8, false>(a, p, ws, stream);
}
