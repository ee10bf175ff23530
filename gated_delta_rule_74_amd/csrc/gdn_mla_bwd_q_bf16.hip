// The bf16 instances of the attention backward: query gradients.
#include "gdn_mla_bwd.hpp"

namespace gdn {
hipError_t launch_mla_bwd_q_bf16(const MlaBwdArgs &a, hipStream_t st) { return mla_bwd_launch<true, true>(a, st); }
} // namespace gdn
