// moe_q4_linear with a scale per 128 columns (kernels in q4.h).
#include "q4.h"

namespace moe {

hipError_t launch_q4_128(const Q4Args &a, hipStream_t st) { return launch_q4_group<128>(a, st); }

}  // namespace moe
