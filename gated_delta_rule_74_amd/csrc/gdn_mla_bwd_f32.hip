// The fp32 instances of the attention backward, and the sum of the shared
// rotary key's gradient over the key heads.
#include "gdn_mla_bwd.hpp"

namespace gdn {

hipError_t launch_mla_bwd_q_f32(const MlaBwdArgs &a, hipStream_t st) { return mla_bwd_launch<false, true>(a, st); }
hipError_t launch_mla_bwd_k_f32(const MlaBwdArgs &a, hipStream_t st) { return mla_bwd_launch<false, false>(a, st); }

// dkr[b,t,hr] = sum over the key heads that share it of their parts, in head
// order; one thread per four columns, read once: bound by the parts' bytes.
template <bool BF> __global__ __launch_bounds__(256) void mla_rope_sum_kernel(MlaBwdArgs a) {
    using S = typename Op<BF>::S;
    const int q = a.s.dr / 4, per = a.s.Hk / a.s.Hr;
    const size_t total = (size_t)a.s.B * a.s.Tk * a.s.Hr * q;
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    const size_t row = i / q; // (b, t, hr)
    const float *p = a.dkr_part + row * per * a.s.dr + (i % q) * 4;
    f32x4 x = zero4();
    for (int h = 0; h < per; ++h) x += *reinterpret_cast<const f32x4 *>(p + (size_t)h * a.s.dr);
    store4((S *)a.dkr + row * a.s.dr + (i % q) * 4, x);
}

hipError_t launch_mla_rope_sum(const MlaBwdArgs &a, bool bf16, hipStream_t st) {
    const size_t total = (size_t)a.s.B * a.s.Tk * a.s.Hr * (a.s.dr / 4);
    const dim3 grid((unsigned)((total + 255) / 256));
    if (bf16) hipLaunchKernelGGL(mla_rope_sum_kernel<true>, grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL(mla_rope_sum_kernel<false>, grid, dim3(256), 0, st, a);
    return hipGetLastError();
}

} // namespace gdn
