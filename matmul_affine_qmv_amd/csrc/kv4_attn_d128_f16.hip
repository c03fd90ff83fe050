// kv4_attn_d128_f16.hip -- attention over the 4-bit cache, head size 128, float16.
#include "kv4_attn_launch.h"

namespace qmx {
namespace kv4 {
template hipError_t launch_dim<128, DT_F16>(const Kv4AttnArgs&, hipStream_t);
}  // namespace kv4
}  // namespace qmx
