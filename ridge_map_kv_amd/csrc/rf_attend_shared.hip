// The attention kernels of bf16 caches whose sequences share prefixes (rf_attend_dev.h).
#include "rf_attend_dev.h"

namespace rf {

template void launch_rows<RF_CACHE_BF16, true>(const AttendArgs&, int, unsigned, hipStream_t);

}  // namespace rf
