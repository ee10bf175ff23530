// Shared prefixes: the fp32 instances (a translation unit of their own, so that the instances compile side by side).
#include "gdn_mla_prefix.hpp"

namespace gdn {
hipError_t launch_mla_prefix_f32(const PrefixArgs &a, hipStream_t st) {
    switch (step_class(a.dl)) {
    case 64: return prefix_run<false, 64, 4, 1>(a, st);
    case 128: return prefix_run<false, 128, 6, 1>(a, st);
    case 192: return prefix_run<false, 192, 8, 1>(a, st);
    case 256: return prefix_run<false, 256, 10, 1>(a, st);
    case 384: return prefix_run<false, 384, 14, 1>(a, st);
    default: return prefix_run<false, 512, 18, 1>(a, st);
    }
}
} // namespace gdn
