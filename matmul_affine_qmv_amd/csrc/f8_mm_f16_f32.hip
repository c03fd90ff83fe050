// 8-bit products into float16, weights' scales in float32.
#include "f8_mm_impl.h"

namespace qmx {
namespace f8 {
void launch_f16_f32(const F8MmArgs& a, F8Plan p, int cus, hipStream_t st) { launch<DT_F16, true>(a, p, cus, st); }
}  // namespace f8
}  // namespace qmx
