// 8-bit products into float16, weights' scales powers of two.
#include "f8_mm_impl.h"

namespace qmx {
namespace f8 {
void launch_f16_e8m0(const F8MmArgs& a, F8Plan p, int cus, hipStream_t st) { launch<DT_F16, false>(a, p, cus, st); }
}  // namespace f8
}  // namespace qmx
