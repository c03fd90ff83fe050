// kv4_attn_d256_bf16.hip -- attention over the 4-bit cache, head size 256, bfloat16.
#include "kv4_attn_launch.h"

namespace qmx {
namespace kv4 {
template hipError_t launch_dim<256, DT_BF16>(const Kv4AttnArgs&, hipStream_t);
}  // namespace kv4
}  // namespace qmx
