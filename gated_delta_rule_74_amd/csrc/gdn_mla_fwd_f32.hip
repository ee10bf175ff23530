// The fp32 instances of the attention forward.
#include "gdn_mla_fwd.hpp"

namespace gdn {
hipError_t launch_mla_fwd_f32(const MlaFwdArgs &a, hipStream_t st) { return mla_fwd_launch<false>(a, st); }
} // namespace gdn
