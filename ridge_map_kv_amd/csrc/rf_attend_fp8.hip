// The attention kernels of caches of e4m3 codes (rf_attend_dev.h).
#include "rf_attend_dev.h"

namespace rf {

template void launch_rows<RF_CACHE_FP8, true>(const AttendArgs&, int, unsigned, hipStream_t);

}  // namespace rf
