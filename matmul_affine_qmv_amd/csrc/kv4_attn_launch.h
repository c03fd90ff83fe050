// kv4_attn_launch.h -- picks the attention kernel of a plan and cache format.
#pragma once

#include "kv4_attn_impl.h"
#include "kv4_prompt_impl.h"

namespace qmx {
namespace kv4 {

template <int D, int GS, int DT>
hipError_t launch_format(const Kv4AttnArgs& a, hipStream_t st) {
    const unsigned groups = (unsigned)(kv4_groups(a));
    if (a.p.rows == PROMPT_ROWS) {
        kv4_prompt_kernel<D, GS, DT><<<groups, 64 * PROMPT_WAVES, 0, st>>>(a);
        return hipGetLastError();
    }
    if constexpr (few_row_waves(D) == 8) {
        if (a.p.waves == 8) {
            kv4_attn_kernel<D, GS, DT, 8><<<groups, 512, 0, st>>>(a);
            return hipGetLastError();
        }
    }
    kv4_attn_kernel<D, GS, DT, 4><<<groups, 256, 0, st>>>(a);
    return hipGetLastError();
}

// One source for each head size and type.
template <int D, int DT>
hipError_t launch_dim(const Kv4AttnArgs& a, hipStream_t st) {
    hipError_t err;
    if (a.c.group == 32) {
        err = launch_format<D, 32, DT>(a, st);
    } else if (D >= 128 && a.c.group == 128) {
        err = launch_format<D, D >= 128 ? 128 : 64, DT>(a, st);
    } else {
        err = launch_format<D, 64, DT>(a, st);
    }
    if (err == hipSuccess && a.p.lines) err = launch_join<D, DT>(a, st);
    return err;
}

extern template hipError_t launch_dim<64, DT_F16>(const Kv4AttnArgs&, hipStream_t);
extern template hipError_t launch_dim<128, DT_F16>(const Kv4AttnArgs&, hipStream_t);
extern template hipError_t launch_dim<256, DT_F16>(const Kv4AttnArgs&, hipStream_t);
extern template hipError_t launch_dim<64, DT_BF16>(const Kv4AttnArgs&, hipStream_t);
extern template hipError_t launch_dim<128, DT_BF16>(const Kv4AttnArgs&, hipStream_t);
extern template hipError_t launch_dim<256, DT_BF16>(const Kv4AttnArgs&, hipStream_t);

}  // namespace kv4
}  // namespace qmx
