// The state after the accepted tokens of a draft: for each of a sequence's
// first counts[n] tokens
//
//   h' = alpha h + k (beta (v - alpha h^T k))^T,  alpha = exp(g A)
//
// (additive: h' = alpha h + k (beta v)^T), the decode step without its output.
// Bound by the state, read and written once: a wave holds 64 columns of one
// head's state in registers, four columns of every fourth row in a lane, so a
// row of the state is read in 16-byte pieces and the sum over the keys ends in
// two exchanges between the wave's quarters. 256 sequences, 16 heads of 56 x 56, up
// to three tokens: 19 us, 5.4 TB/s; 33 sequences, 8 heads of 64 x 64, up to seven: 10 us,
// the chain of the tokens.
#include "gdn_common.hpp"
#include "gdn_serve.hpp"

namespace gdn {

constexpr int CW = 4; // waves of a workgroup

// Four columns of a row that has `left` more of them (at least one); what
// stands in place of those past its end is not used.
template <bool VEC> __device__ __forceinline__ f32x4 load4(const float *p, int left) {
    if constexpr (VEC) return *reinterpret_cast<const f32x4 *>(p);
    f32x4 x;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = p[min(e, left - 1)];
    return x;
}
template <bool VEC> __device__ __forceinline__ f32x4 load4(const u16 *p, int left) {
    if constexpr (VEC) {
        const uint2 w = *reinterpret_cast<const uint2 *>(p);
        return f32x4{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xffff0000u)};
    }
    f32x4 x;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = bf2f(p[min(e, left - 1)]);
    return x;
}

// RI: state rows of a lane (a quarter of the padded key width)
template <bool BF, int RI, bool VEC> __global__ __launch_bounds__(CW * 64) void commit_kernel(CommitArgs a) {
    using S = typename Op<BF>::S;
    __shared__ __align__(16) float ks[CW][4 * RI];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, quarter = lane >> 4;
    const int blocks = (a.dv + 63) / 64;
    const long long item = (long long)blockIdx.x * CW + wave;
    if (item >= (long long)a.N * a.H * blocks) return;
    const int nh = (int)(item / blocks), first = (int)(item % blocks) * 64, mine = first + 4 * (lane & 15);
    const int n = nh / a.H, h = nh % a.H, dk = a.dk, dv = a.dv;
    // (lanes past the last column work on the first ones again and store nothing)
    const bool ok = mine < dv;
    const int c0 = ok ? mine : first, left = dv - c0;
    const int count = min(max(a.counts[n], 0), a.S);
    if (count == 0 && a.h_in == a.h_out) return;
    const size_t at = (size_t)nh * dk * dv + c0;
    f32x4 x[RI];
#pragma unroll
    for (int i = 0; i < RI; ++i) x[i] = zero4();
    if (a.h_in) {
#pragma unroll
        for (int i = 0; i < RI; ++i) {
            if (4 * i >= dk) continue;
            const int row = 4 * i + quarter; // (rows past dk: zero, their keys are)
            const f32x4 y = load4<VEC>(a.h_in + at + (size_t)min(row, dk - 1) * dv, left);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i][e] = row < dk ? y[e] : 0.f;
        }
    }
    const float A = -expf(a.A_log[h]);
    float *kw = ks[wave];
    for (int t = 0; t < count; ++t) {
        const size_t tok = ((size_t)n * a.S + t) * a.H + h;
        const S *kp = (const S *)a.k + tok * dk;
        const float alpha = expf(gate_of(a.g[tok], a.logits) * A), beta = gate_of(a.beta[tok], a.logits);
        const f32x4 v = load4<VEC>((const S *)a.v + tok * dv + c0, left);
        float ka = lane < dk ? to_f(kp[lane]) : 0.f, kb = RI > 16 && lane + 64 < dk ? to_f(kp[lane + 64]) : 0.f;
        if (a.l2k) { // k / sqrt(|k|^2 + KEY_EPS)
            float ss = ka * ka + kb * kb;
#pragma unroll
            for (int off = 32; off > 0; off >>= 1) ss += __shfl_xor(ss, off, 64);
            const float inv = 1.f / sqrtf(ss + KEY_EPS);
            ka *= inv;
            kb *= inv;
        }
        // key j where its quarter reads its rows' keys one after the other; the
        // wave reads back only what it wrote: no barrier beyond the wave's
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        kw[(lane & 3) * RI + (lane >> 2)] = ka;
        if (RI > 16) kw[(lane & 3) * RI + 16 + (lane >> 2)] = kb;
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        const float *kq = kw + quarter * RI;
        f32x4 w = v * beta;
        if (!a.additive) {
            f32x4 u = zero4();
#pragma unroll
            for (int i = 0; i < RI; i += 4) {
                const f32x4 k4 = *reinterpret_cast<const f32x4 *>(kq + i);
#pragma unroll
                for (int e = 0; e < 4; ++e) u += x[i + e] * k4[e];
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = beta * (v[e] - alpha * sum4g(u[e]));
        }
#pragma unroll
        for (int i = 0; i < RI; i += 4) {
            const f32x4 k4 = *reinterpret_cast<const f32x4 *>(kq + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i + e] = x[i + e] * alpha + w * k4[e];
        }
    }
#pragma unroll
    for (int i = 0; i < RI; ++i) {
        const int row = 4 * i + quarter;
        if (row >= dk || !ok) continue;
        float *p = a.h_out + at + (size_t)row * dv;
        if constexpr (VEC) {
            store4(p, x[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < left) p[e] = x[i][e];
        }
    }
}

long long step_commit_groups(int N, int H, int dv) { return ((long long)N * H * ((dv + 63) / 64) + CW - 1) / CW; }
template <bool BF, int RI> static hipError_t commit_run(const CommitArgs &a, hipStream_t st) {
    const dim3 grid((unsigned)step_commit_groups(a.N, a.H, a.dv));
    // 16-byte pieces where every row of the state and of v begins on one
    const auto on = [](const void *p, size_t n) { return (uintptr_t)p % n == 0; };
    if (a.dv % 4 == 0 && on(a.h_in, 16) && on(a.h_out, 16) && on(a.v, BF ? 8 : 16))
        hipLaunchKernelGGL((commit_kernel<BF, RI, true>), grid, dim3(CW * 64), 0, st, a);
    else hipLaunchKernelGGL((commit_kernel<BF, RI, false>), grid, dim3(CW * 64), 0, st, a);
    return hipGetLastError();
}
hipError_t launch_step_commit(const CommitArgs &a, bool bf16, hipStream_t st) {
    if (a.dk <= 64) return bf16 ? commit_run<true, 16>(a, st) : commit_run<false, 16>(a, st);
    return bf16 ? commit_run<true, 32>(a, st) : commit_run<false, 32>(a, st);
}

} // namespace gdn
