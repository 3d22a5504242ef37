// moe_q4_linear with a scale per 64 columns (kernels in q4.h).
#include "q4.h"

namespace moe {

hipError_t launch_q4_64(const Q4Args &a, hipStream_t st) { return launch_q4_group<64>(a, st); }

}  // namespace moe
