// Per-head RMS norm and position rotation in one pass, its backward, and the
// write of new tokens' latents and rotary keys into the paged cache.
//
//   z = x / sqrt(mean(x^2) + eps) * w,   y = z with the last r columns turned:
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = pos * freqs[i]
//
// for the pairs (i, i + r/2) of the turned columns, or (2i, 2i + 1) when
// interleaved. All of it is bound by the bytes of x and y: a row (token, head)
// is held by LPR lanes, eight columns each, in one read and one write; the
// norm's sum goes over those lanes; a pair's other half is read again (it is
// in L1). The sine and cosine of a token are formed once for all its heads, in
// LDS. The angle is the product of position and frequency in fp64, reduced to
// a fraction of a turn there, so that far positions lose nothing.
#include "gdn_mla.hpp"

namespace gdn {

constexpr int NR_THREADS = 256, NR_PAIRS = 1024; // (LPR >= d / 8, so 256 / LPR rows hold at most 1024 pairs)

__device__ __forceinline__ float2 turn_of(int pos, double freq) {
    double t = (double)pos * freq * 0.15915494309189533577; // turns
    t -= rint(t);
    float2 cs;
    sincospif(2.f * (float)t, &cs.y, &cs.x);
    return cs;
}

__device__ __forceinline__ float lanes_sum(float x, int lpr) {
    for (int o = lpr >> 1; o >= 1; o >>= 1) x += __shfl_xor(x, o, 64);
    return x;
}

// How a row's columns lie on its lanes: eight consecutive ones each (VEC: 16-
// byte accesses, every pair whole in a vector or a vector's distance apart),
// or lane + LPR * j.
template <bool VEC> __device__ __forceinline__ int col_of(int sub, int j, int lpr) {
    return VEC ? sub * 8 + j : sub + lpr * j;
}
template <bool BF, bool VEC>
__device__ __forceinline__ void load_row(const typename Op<BF>::S *x, int sub, int lpr, int d, bool in, float *v) {
    using S = typename Op<BF>::S;
    if constexpr (VEC) {
        const bool on = in && sub * 8 < d;
        S s[8];
        if constexpr (BF) {
            *reinterpret_cast<uint4 *>(s) = on ? *reinterpret_cast<const uint4 *>(x + sub * 8) : uint4{0u, 0u, 0u, 0u};
        } else {
            *reinterpret_cast<f32x4 *>(s) = on ? *reinterpret_cast<const f32x4 *>(x + sub * 8) : zero4();
            *reinterpret_cast<f32x4 *>(s + 4) = on ? *reinterpret_cast<const f32x4 *>(x + sub * 8 + 4) : zero4();
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = to_f(s[j]);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = in && sub + lpr * j < d ? to_f(x[sub + lpr * j]) : 0.f;
    }
}
template <bool BF, bool VEC>
__device__ __forceinline__ void store_row(typename Op<BF>::S *y, int sub, int lpr, int d, const float *v) {
    using S = typename Op<BF>::S;
    if constexpr (VEC) {
        if (sub * 8 >= d) return;
        store4(y + sub * 8, f32x4{v[0], v[1], v[2], v[3]});
        store4(y + sub * 8 + 4, f32x4{v[4], v[5], v[6], v[7]});
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (sub + lpr * j < d) y[sub + lpr * j] = from_f<BF>(v[j]);
    }
}

// The column turned against column c (in the last r ones) and the pair's index.
__device__ __forceinline__ int partner(int c, int d, int r, bool inter, int &pair, bool &second) {
    const int p = c - (d - r);
    if (inter) {
        pair = p >> 1;
        second = p & 1;
        return second ? c - 1 : c + 1;
    }
    second = p >= r / 2;
    pair = second ? p - r / 2 : p;
    return second ? c - r / 2 : c + r / 2;
}

// v (already scaled by w) turned by sign * angle. raw: the row before scaling
// by `f` (and w); in: the row exists.
template <bool BF, bool VEC>
__device__ __forceinline__ void turn_row(float *v, const typename Op<BF>::S *raw, const float *w, float f, int sub,
                                         int lpr, int d, int r, bool inter, float sign, const float2 *cs, bool in) {
    if (r == 0) return;
    if (VEC && inter) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const int c = sub * 8 + j;
            if (c < d - r || c >= d) continue;
            const float2 t = cs[(c - (d - r)) >> 1];
            const float a = v[j], b = v[j + 1], sn = sign * t.y;
            v[j] = a * t.x - b * sn;
            v[j + 1] = b * t.x + a * sn;
        }
        return;
    }
    if (VEC) {
        const int c0 = sub * 8;
        if (c0 < d - r || c0 >= d) return;
        int pair;
        bool second;
        const int pc = partner(c0, d, r, false, pair, second);
        float o[8];
        load_row<BF, true>(raw + pc, 0, 1, 8, in, o);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 t = cs[pair + j];
            const float b = o[j] * f * (w ? w[pc + j] : 1.f);
            v[j] = v[j] * t.x + (second ? sign : -sign) * b * t.y;
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = sub + lpr * j;
        if (c < d - r || c >= d) continue;
        int pair;
        bool second;
        const int pc = partner(c, d, r, inter, pair, second);
        const float b = (in ? to_f(raw[pc]) : 0.f) * f * (w ? w[pc] : 1.f);
        v[j] = v[j] * cs[pair].x + (second ? sign : -sign) * b * cs[pair].y;
    }
}

// The turns of the tokens of rows row0 .. row0 + rpp - 1.
__device__ __forceinline__ void fill_turns(const NormRopeArgs &a, float2 *cs, long long row0, int rpp, long long rows) {
    const int hp = a.r / 2;
    if (hp == 0) return;
    const long long t0 = row0 / a.H, t1 = (min(row0 + rpp, rows) - 1) / a.H;
    for (int e = threadIdx.x; e < (int)(t1 - t0 + 1) * hp; e += NR_THREADS)
        cs[e] = turn_of(a.pos[t0 + e / hp], a.freqs[e % hp]);
}

template <bool BF, bool VEC> __global__ __launch_bounds__(NR_THREADS) void norm_rope_kernel(NormRopeArgs a, int lpr) {
    using S = typename Op<BF>::S;
    __shared__ float2 cs[NR_PAIRS];
    const int rpp = NR_THREADS / lpr, sub = threadIdx.x % lpr, d = a.d;
    const long long rows = a.M * a.H;
    for (long long row0 = (long long)blockIdx.x * rpp; row0 < rows; row0 += (long long)gridDim.x * rpp) {
        const long long row = row0 + threadIdx.x / lpr;
        const bool in = row < rows;
        const S *x = (const S *)a.x + (in ? row : 0) * d;
        float v[8];
        load_row<BF, VEC>(x, sub, lpr, d, in, v);
        fill_turns(a, cs, row0, rpp, rows);
        float inv = 1.f;
        if (a.norm) {
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
            inv = 1.f / sqrtf(lanes_sum(ss, lpr) / (float)d + a.eps);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int c = col_of<VEC>(sub, j, lpr);
            v[j] *= inv * (a.w && c < d ? a.w[c] : 1.f);
        }
        __syncthreads();
        const float2 *t = cs + (a.r / 2) * (int)((in ? row : row0) / a.H - row0 / a.H);
        turn_row<BF, VEC>(v, x, a.w, inv, sub, lpr, d, a.r, a.inter, 1.f, t, in);
        if (in) store_row<BF, VEC>((S *)a.y + row * d, sub, lpr, d, v);
        __syncthreads();
    }
}

// Backward: dz = dy turned back, xh = x inv,
//   dx = inv (dz w - xh mean(dz w xh)),   dw = sum over rows of dz xh
// A thread keeps the same columns over all its rows and so sums its part of dw
// in registers; the parts of a workgroup's row slots are added in slot order,
// those of the workgroups by norm_sum_kernel: a fixed order throughout.
template <bool BF, bool VEC> __global__ __launch_bounds__(NR_THREADS) void norm_rope_bwd_kernel(NormRopeArgs a, int lpr) {
    using S = typename Op<BF>::S;
    __shared__ float2 cs[NR_PAIRS];
    __shared__ float red[NR_THREADS * 8];
    const int rpp = NR_THREADS / lpr, sub = threadIdx.x % lpr, d = a.d;
    const long long rows = a.M * a.H;
    float dw[8] = {};
    for (long long row0 = (long long)blockIdx.x * rpp; row0 < rows; row0 += (long long)gridDim.x * rpp) {
        const long long row = row0 + threadIdx.x / lpr;
        const bool in = row < rows;
        const S *dy = (const S *)a.dy + (in ? row : 0) * d;
        float v[8], x[8] = {};
        load_row<BF, VEC>(dy, sub, lpr, d, in, v);
        if (a.norm) load_row<BF, VEC>((const S *)a.x + (in ? row : 0) * d, sub, lpr, d, in, x);
        fill_turns(a, cs, row0, rpp, rows);
        __syncthreads();
        const float2 *t = cs + (a.r / 2) * (int)((in ? row : row0) / a.H - row0 / a.H);
        turn_row<BF, VEC>(v, dy, nullptr, 1.f, sub, lpr, d, a.r, a.inter, -1.f, t, in);
        if (a.norm) {
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
            const float inv = 1.f / sqrtf(lanes_sum(ss, lpr) / (float)d + a.eps);
            float dot = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = col_of<VEC>(sub, j, lpr);
                x[j] *= inv;
                dw[j] = fmaf(v[j], x[j], dw[j]);
                v[j] *= a.w && c < d ? a.w[c] : 1.f;
                dot = fmaf(v[j], x[j], dot);
            }
            dot = lanes_sum(dot, lpr) / (float)d;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = inv * (v[j] - x[j] * dot);
        }
        if (in) store_row<BF, VEC>((S *)a.y + row * d, sub, lpr, d, v);
        __syncthreads();
    }
    if (!a.dw) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) red[threadIdx.x * 8 + j] = dw[j];
    __syncthreads();
    for (int c = threadIdx.x; c < d; c += NR_THREADS) {
        const int sl = VEC ? c / 8 : c % lpr, j = VEC ? c % 8 : c / lpr;
        float x = 0.f;
        for (int k = 0; k < rpp; ++k) x += red[(k * lpr + sl) * 8 + j];
        a.dw_part[(size_t)blockIdx.x * d + c] = x;
    }
}

// dw[c] = sum of the workgroups' parts; a workgroup takes 16 columns, 16
// threads along the parts of each, in a fixed order.
__global__ __launch_bounds__(256) void norm_sum_kernel(NormRopeArgs a) {
    __shared__ float red[16][17];
    const int c = blockIdx.x * 16 + (threadIdx.x & 15), k = threadIdx.x >> 4;
    float x = 0.f;
    if (c < a.d)
        for (int b = k; b < a.nblk; b += 16) x += a.dw_part[(size_t)b * a.d + c];
    red[k][threadIdx.x & 15] = x;
    __syncthreads();
    if (k == 0 && c < a.d) {
        for (int i = 1; i < 16; ++i) x += red[i][threadIdx.x];
        a.dw[c] = x;
    }
}

static int lanes_per_row(int d) {
    int l = 1;
    while (l * 8 < d) l *= 2;
    return l;
}
// Every pair lies in one 8-column vector, or the halves are whole vectors apart.
static bool row_vectors(int d, int r, int inter) {
    return d % 8 == 0 && (r == 0 || inter || (r % 16 == 0 && (d - r) % 8 == 0));
}
static long long passes(long long rows, int d) {
    const int rpp = NR_THREADS / lanes_per_row(d);
    return (rows + rpp - 1) / rpp;
}
int norm_rope_blocks(long long rows, int d) {
    const long long p = passes(rows, d);
    return p < 1024 ? (int)p : 1024;
}

hipError_t launch_norm_rope(const NormRopeArgs &a, bool bf16, hipStream_t st) {
    const int lpr = lanes_per_row(a.d);
    const long long p = passes(a.M * a.H, a.d);
    const dim3 grid((unsigned)(p < 16384 ? p : 16384));
    const bool vec = row_vectors(a.d, a.r, a.inter);
    if (bf16 && vec) hipLaunchKernelGGL((norm_rope_kernel<true, true>), grid, dim3(NR_THREADS), 0, st, a, lpr);
    else if (bf16) hipLaunchKernelGGL((norm_rope_kernel<true, false>), grid, dim3(NR_THREADS), 0, st, a, lpr);
    else if (vec) hipLaunchKernelGGL((norm_rope_kernel<false, true>), grid, dim3(NR_THREADS), 0, st, a, lpr);
    else hipLaunchKernelGGL((norm_rope_kernel<false, false>), grid, dim3(NR_THREADS), 0, st, a, lpr);
    return hipGetLastError();
}
hipError_t launch_norm_rope_bwd(const NormRopeArgs &a, bool bf16, hipStream_t st) {
    const int lpr = lanes_per_row(a.d);
    const dim3 grid((unsigned)a.nblk);
    const bool vec = row_vectors(a.d, a.r, a.inter);
    if (bf16 && vec) hipLaunchKernelGGL((norm_rope_bwd_kernel<true, true>), grid, dim3(NR_THREADS), 0, st, a, lpr);
    else if (bf16) hipLaunchKernelGGL((norm_rope_bwd_kernel<true, false>), grid, dim3(NR_THREADS), 0, st, a, lpr);
    else if (vec) hipLaunchKernelGGL((norm_rope_bwd_kernel<false, true>), grid, dim3(NR_THREADS), 0, st, a, lpr);
    else hipLaunchKernelGGL((norm_rope_bwd_kernel<false, false>), grid, dim3(NR_THREADS), 0, st, a, lpr);
    return hipGetLastError();
}
hipError_t launch_norm_sum(const NormRopeArgs &a, hipStream_t st) {
    hipLaunchKernelGGL(norm_sum_kernel, dim3((unsigned)((a.d + 15) / 16)), dim3(256), 0, st, a);
    return hipGetLastError();
}

// A new token's cache row: its latent normalised, its rotary key turned, at
// the slot the plan gave it. One group of LPR lanes per token; each pair's
// turn is needed once, so it is formed where it is used. Slots outside the
// pool (-1: none) are skipped.
template <bool BF> __global__ __launch_bounds__(NR_THREADS) void mla_write_kernel(MlaWriteArgs a, int lpr) {
    using S = typename Op<BF>::S;
    const int sub = threadIdx.x % lpr;
    const long long i = (long long)blockIdx.x * (NR_THREADS / lpr) + threadIdx.x / lpr;
    const int slot = i < a.n ? a.slots[i] : -1;
    const bool in = slot >= 0 && slot < a.n_slots; // (the whole group takes part in the sum below)
    float v[8];
    load_row<BF, true>((const S *)a.c + (in ? i : 0) * a.dl, sub, lpr, a.dl, in, v);
    float inv = 1.f;
    if (a.norm) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
        inv = 1.f / sqrtf(lanes_sum(ss, lpr) / (float)a.dl + a.eps);
    }
    if (!in) return;
    S *row = (S *)a.cache + (size_t)slot * (a.dl + a.dr);
    if (sub * 8 < a.dl) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= inv * (a.w ? a.w[sub * 8 + j] : 1.f);
        store_row<BF, true>(row, sub, lpr, a.dl, v);
    }
    const S *kr = (const S *)a.kr + i * a.dr;
    const int hp = a.dr / 2;
    for (int p = sub; p < hp; p += lpr) {
        const int ca = a.inter ? 2 * p : p, cb = a.inter ? 2 * p + 1 : p + hp;
        const float x = to_f(kr[ca]), y = to_f(kr[cb]);
        const float2 t = a.freqs ? turn_of(a.pos[i], a.freqs[p]) : float2{1.f, 0.f};
        row[a.dl + ca] = from_f<BF>(x * t.x - y * t.y);
        row[a.dl + cb] = from_f<BF>(y * t.x + x * t.y);
    }
}

hipError_t launch_mla_write(const MlaWriteArgs &a, bool bf16, hipStream_t st) {
    int lpr = lanes_per_row(a.dl);
    if (lpr < 8) lpr = 8; // (narrow latents: the lanes share the pairs)
    const int per = NR_THREADS / lpr;
    const dim3 grid((unsigned)((a.n + per - 1) / per));
    if (bf16) hipLaunchKernelGGL(mla_write_kernel<true>, grid, dim3(NR_THREADS), 0, st, a, lpr);
    else hipLaunchKernelGGL(mla_write_kernel<false>, grid, dim3(NR_THREADS), 0, st, a, lpr);
    return hipGetLastError();
}

} // namespace gdn
