// The bf16 instances of the attention forward (a translation unit of their
// own, so that the instances compile side by side).
#include "gdn_mla_fwd.hpp"

namespace gdn {
MlaPad mla_pad(const MlaArgs &s) {
    const int d = s.dn + s.dr;
    if (d <= 32 && s.dv <= 32) return {32, 32};
    return {d <= 64 ? 64 : d <= 96 ? 96 : d <= 128 ? 128 : 192, s.dv <= 64 ? 64 : 128};
}
hipError_t launch_mla_fwd_bf16(const MlaFwdArgs &a, hipStream_t st) { return mla_fwd_launch<true>(a, st); }
} // namespace gdn
