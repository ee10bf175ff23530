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
// in L1, asked for together with the first). The sine and cosine of a token are
// formed once for all its heads, in LDS. B8 T4096 H16 d88 bf16: forward 49 us
// (3.8 TB/s), backward 60 us (4.6 TB/s) and 6 us for dw's sum, where a large
// copy reaches 5.6. The angle is the product of position and frequency in fp64, reduced to
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

// Sum over the lpr lanes of a row (a power of two), every lane gets it: moves
// inside a 16-lane row, then between rows, none through LDS.
__device__ __forceinline__ float lanes_sum(float x, int lpr) {
    if (lpr >= 2) x += dpp_f<0xB1>(x);   // lane ^ 1
    if (lpr >= 4) x += dpp_f<0x4E>(x);   // lane ^ 2
    if (lpr >= 8) x += dpp_f<0x141>(x);  // mirrored within 8
    if (lpr >= 16) x += dpp_f<0x140>(x); // mirrored within 16
    if (lpr >= 32) {
        const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    }
    if (lpr >= 64) {
        const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(p[0]) + __uint_as_float(p[1]);
    }
    return x;
}

// How a row's columns lie on its lanes: eight consecutive ones each (VEC: 16-
// byte accesses, every pair whole in a vector or a vector's distance apart),
// or lane + LPR * j.
template <bool VEC> __device__ __forceinline__ int col_of(int sub, int j, int lpr) {
    return VEC ? sub * 8 + j : sub + lpr * j;
}

// A lane's eight values of a row, as loaded; zeros where there is none.
template <bool BF, bool VEC> struct Raw {
    using S = typename Op<BF>::S;
    u32x4 q[VEC ? (BF ? 1 : 2) : 1];
    S s[VEC ? 1 : 8];
    __device__ __forceinline__ void load(const S *x, int sub, int lpr, int d, bool in) {
        if constexpr (VEC) {
            const void *p = in && sub * 8 < d ? (const void *)(x + sub * 8) : (const void *)&mla_zeros;
            q[0] = load16(p);
            if constexpr (!BF) q[1] = load16(in && sub * 8 < d ? (const void *)(x + sub * 8 + 4) : (const void *)&mla_zeros);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] = in && sub + lpr * j < d ? x[sub + lpr * j] : S(0);
        }
    }
    __device__ __forceinline__ void values(float *v) const {
        if constexpr (VEC && BF) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = __uint_as_float(q[0][j] << 16);
                v[2 * j + 1] = __uint_as_float(q[0][j] & 0xffff0000u);
            }
        } else if constexpr (VEC) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(q[j / 4][j % 4]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = to_f(s[j]);
        }
    }
};
template <bool BF, bool VEC>
__device__ __forceinline__ void store_row(typename Op<BF>::S *y, int sub, int lpr, int d, const float *v) {
    if constexpr (VEC) {
        if (sub * 8 >= d) return;
        if constexpr (BF) {
            uint4 w;
            w.x = f2bf2(v[0], v[1]);
            w.y = f2bf2(v[2], v[3]);
            w.z = f2bf2(v[4], v[5]);
            w.w = f2bf2(v[6], v[7]);
            *reinterpret_cast<uint4 *>(y + sub * 8) = w;
        } else {
            store4(y + sub * 8, f32x4{v[0], v[1], v[2], v[3]});
            store4(y + sub * 8 + 4, f32x4{v[4], v[5], v[6], v[7]});
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (sub + lpr * j < d) y[sub + lpr * j] = from_f<BF>(v[j]);
    }
}

// What a lane's columns have to do with the turn: fixed over all rows.
//   VEC, interleaved: pairs (j, j + 1) of the lane itself, from pair `pair` on;
//   VEC, halves: the eight columns `other` hold the pairs' other halves;
//   else: each column by itself (part()).
template <bool VEC> struct Turn {
    bool any, second;
    int other, pair;
    __device__ __forceinline__ Turn(const NormRopeArgs &a, int sub) {
        const int c = sub * 8 - (a.d - a.r); // first column, from the first turned one
        any = VEC && a.r > 0 && c >= 0 && sub * 8 < a.d;
        second = !a.inter && c >= a.r / 2;
        pair = a.inter ? c / 2 : second ? c - a.r / 2 : c;
        other = second ? sub * 8 - a.r / 2 : sub * 8 + a.r / 2;
    }
    // a single column's partner, pair and half
    __device__ static __forceinline__ int part(const NormRopeArgs &a, int c, int &pair, bool &second) {
        const int p = c - (a.d - a.r);
        if (a.inter) {
            pair = p >> 1;
            second = p & 1;
            return second ? c - 1 : c + 1;
        }
        second = p >= a.r / 2;
        pair = second ? p - a.r / 2 : p;
        return second ? c - a.r / 2 : c + a.r / 2;
    }
};

// v turned by sign * angle (cs: cosine and sine of the token's pairs). o: the
// other halves of a VEC lane's pairs; raw, f, w: for the rest, the row they are
// read from and what scales them.
template <bool BF, bool VEC>
__device__ __forceinline__ void turn_row(const NormRopeArgs &a, const Turn<VEC> &tn, float *v, const float *o,
                                         const typename Op<BF>::S *raw, float f, const float *w, int sub, int lpr,
                                         float sign, const float2 *cs, bool in) {
    if constexpr (VEC) {
        if (!tn.any) return;
        if (a.inter) {
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float2 t = cs[tn.pair + j / 2];
                const float x = v[j], y = v[j + 1], sn = sign * t.y;
                v[j] = x * t.x - y * sn;
                v[j + 1] = y * t.x + x * sn;
            }
        } else {
            const float sg = tn.second ? sign : -sign;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float2 t = cs[tn.pair + j];
                v[j] = v[j] * t.x + sg * o[j] * t.y;
            }
        }
        return;
    }
    if (a.r == 0) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = sub + lpr * j;
        if (c < a.d - a.r || c >= a.d) continue;
        int pair;
        bool second;
        const int pc = Turn<VEC>::part(a, c, pair, second);
        const float b = (in ? to_f(raw[pc]) : 0.f) * f * (w ? w[pc] : 1.f);
        v[j] = v[j] * cs[pair].x + (second ? sign : -sign) * b * cs[pair].y;
    }
}

// The turns of the tokens of rows row0 .. row0 + rpp - 1.
__device__ __forceinline__ void fill_turns(const NormRopeArgs &a, float2 *cs, unsigned row0, unsigned rpp, unsigned rows) {
    const int hp = a.r / 2;
    if (hp == 0) return;
    const unsigned t0 = row0 / (unsigned)a.H, t1 = (min(row0 + rpp, rows) - 1) / (unsigned)a.H;
    for (int e = threadIdx.x; e < (int)(t1 - t0 + 1) * hp; e += NR_THREADS)
        cs[e] = turn_of(a.pos[t0 + e / hp], a.freqs[e % hp]);
}

// UN rows per thread and pass, all requested before the first is used: with
// one row the kernel waits for memory most of the time (B8 T4096 H16 d88 bf16:
// 130 us with one row in flight per thread).
template <bool BF, bool VEC, int UN>
__global__ __launch_bounds__(NR_THREADS) void norm_rope_kernel(NormRopeArgs a, int lpr) {
    using S = typename Op<BF>::S;
    __shared__ float2 cs[2][NR_PAIRS];
    const int sub = threadIdx.x % lpr, d = a.d;
    const unsigned slots = NR_THREADS / lpr, rpp = slots * UN;
    const unsigned rows = (unsigned)(a.M * a.H); // (x has fewer than 2^31 elements)
    const float per_d = 1.f / (float)d;
    const Turn<VEC> tn(a, sub);
    const bool halves = tn.any && !a.inter;
    float w[8], wo[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = col_of<VEC>(sub, j, lpr);
        w[j] = a.w && c < d ? a.w[c] : 1.f;
        wo[j] = a.w && halves ? a.w[tn.other + j] : 1.f;
    }
    int buf = 0;
    for (unsigned row0 = blockIdx.x * rpp; row0 < rows; row0 += gridDim.x * rpp, buf ^= 1) {
        const unsigned first = row0 + threadIdx.x / lpr, token0 = row0 / (unsigned)a.H;
        Raw<BF, VEC> x[UN], o[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const unsigned row = first + u * slots;
            const S *p = (const S *)a.x + (size_t)(row < rows ? row : 0) * d;
            x[u].load(p, sub, lpr, d, row < rows);
            if (VEC) o[u].load(p + (halves ? tn.other - sub * 8 : 0), sub, lpr, d, row < rows && halves);
        }
        fill_turns(a, cs[buf], row0, rpp, rows);
        __syncthreads(); // (the other table's last readers passed here too)
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const unsigned row = first + u * slots;
            const bool in = row < rows;
            float v[8], ov[8];
            x[u].values(v);
            float inv = 1.f;
            if (a.norm) {
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
                inv = rsqrtf(fmaf(lanes_sum(ss, lpr), per_d, a.eps));
            }
            if (VEC) o[u].values(ov);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] *= inv * w[j];
                if (VEC) ov[j] *= inv * wo[j];
            }
            const float2 *t = cs[buf] + (a.r / 2) * ((in ? row : row0) / (unsigned)a.H - token0);
            turn_row<BF, VEC>(a, tn, v, ov, (const S *)a.x + (size_t)(in ? row : 0) * d, inv, a.w, sub, lpr, 1.f, t, in);
            // y may be x: where a column's partner is read from memory, every lane of the row has read before
            // any writes (a row's lanes are in one wave)
            if (!VEC) __builtin_amdgcn_wave_barrier();
            if (in) store_row<BF, VEC>((S *)a.y + (size_t)row * d, sub, lpr, d, v);
        }
    }
}

// Backward: dz = dy turned back, xh = x inv,
//   dx = inv (dz w - xh mean(dz w xh)),   dw = sum over rows of dz xh
// A thread keeps the same columns over all its rows and so sums its part of dw
// in registers; the parts of a workgroup's row slots are added in slot order,
// those of the workgroups by norm_sum_kernel: a fixed order throughout.
template <bool BF, bool VEC, int UN>
__global__ __launch_bounds__(NR_THREADS) void norm_rope_bwd_kernel(NormRopeArgs a, int lpr) {
    using S = typename Op<BF>::S;
    __shared__ float2 cs[2][NR_PAIRS];
    __shared__ float red[NR_THREADS * 8];
    const int sub = threadIdx.x % lpr, d = a.d;
    const unsigned slots = NR_THREADS / lpr, rpp = slots * UN;
    const unsigned rows = (unsigned)(a.M * a.H); // (x has fewer than 2^31 elements)
    const float per_d = 1.f / (float)d;
    const Turn<VEC> tn(a, sub);
    const bool halves = tn.any && !a.inter;
    float w[8], dw[8] = {};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int c = col_of<VEC>(sub, j, lpr);
        w[j] = a.w && c < d ? a.w[c] : 1.f;
    }
    int buf = 0;
    for (unsigned row0 = blockIdx.x * rpp; row0 < rows; row0 += gridDim.x * rpp, buf ^= 1) {
        const unsigned first = row0 + threadIdx.x / lpr, token0 = row0 / (unsigned)a.H;
        Raw<BF, VEC> g[UN], o[UN], x[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const unsigned row = first + u * slots;
            const size_t at = (size_t)(row < rows ? row : 0) * d;
            const S *p = (const S *)a.dy + at;
            g[u].load(p, sub, lpr, d, row < rows);
            if (VEC) o[u].load(p + (halves ? tn.other - sub * 8 : 0), sub, lpr, d, row < rows && halves);
            if (a.norm) x[u].load((const S *)a.x + at, sub, lpr, d, row < rows);
        }
        fill_turns(a, cs[buf], row0, rpp, rows);
        __syncthreads();
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const unsigned row = first + u * slots;
            const bool in = row < rows;
            float v[8], ov[8];
            g[u].values(v);
            if (VEC) o[u].values(ov);
            const float2 *t = cs[buf] + (a.r / 2) * ((in ? row : row0) / (unsigned)a.H - token0);
            turn_row<BF, VEC>(a, tn, v, ov, (const S *)a.dy + (size_t)(in ? row : 0) * d, 1.f, nullptr, sub, lpr, -1.f, t, in);
            if (a.norm) {
                float xh[8], ss = 0.f;
                x[u].values(xh);
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(xh[j], xh[j], ss);
                const float inv = rsqrtf(fmaf(lanes_sum(ss, lpr), per_d, a.eps));
                float dot = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    xh[j] *= inv;
                    dw[j] = fmaf(v[j], xh[j], dw[j]);
                    v[j] *= w[j];
                    dot = fmaf(v[j], xh[j], dot);
                }
                dot = lanes_sum(dot, lpr) * per_d;
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = inv * (v[j] - xh[j] * dot);
            }
            if (in) store_row<BF, VEC>((S *)a.y + (size_t)row * d, sub, lpr, d, v);
        }
    }
    if (!a.dw) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) red[threadIdx.x * 8 + j] = dw[j];
    __syncthreads();
    for (int c = threadIdx.x; c < d; c += NR_THREADS) {
        const int sl = VEC ? c / 8 : c % lpr, j = VEC ? c % 8 : c / lpr;
        float x = 0.f;
        for (unsigned k = 0; k < slots; ++k) x += red[(k * lpr + sl) * 8 + j];
        a.dw_part[(size_t)blockIdx.x * d + c] = x;
    }
}

// dw[c] = sum of the workgroups' parts, in a fixed order: a workgroup takes
// four columns, thread t the parts t, t + 256, ..., then the threads in halves.
__global__ __launch_bounds__(256) void norm_sum_kernel(NormRopeArgs a) {
    __shared__ __align__(16) float red[256][4];
    const int c0 = blockIdx.x * 4, t = threadIdx.x;
    float x[4] = {};
    for (int b = t; b < a.nblk; b += 256) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (c0 + k < a.d) x[k] += a.dw_part[(size_t)b * a.d + c0 + k];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) red[t][k] = x[k];
    for (int o = 128; o >= 1; o >>= 1) {
        __syncthreads();
        if (t < o) {
#pragma unroll
            for (int k = 0; k < 4; ++k) red[t][k] += red[t + o][k];
        }
    }
    if (t < 4 && c0 + t < a.d) a.dw[c0 + t] = red[0][t];
}

static int lanes_per_row(int d) {
    int l = 1;
    while (l * 8 < d) l *= 2;
    return l;
}
// The turned columns begin with a vector, and every pair lies in one vector
// (interleaved: vectors are of even length) or its halves are whole vectors apart.
static bool row_vectors(int d, int r, int inter) {
    return d % 8 == 0 && (r == 0 || ((d - r) % 8 == 0 && (inter || r % 16 == 0)));
}
static long long passes(long long rows, int d, int un) {
    const int rpp = NR_THREADS / lanes_per_row(d) * un;
    return (rows + rpp - 1) / rpp;
}
// Rows per thread: four once that still leaves a workgroup for every CU and
// the turns of a pass's tokens fit the table.
static int rows_per_thread(const NormRopeArgs &a, bool vec) {
    const int rpp = NR_THREADS / lanes_per_row(a.d) * 4;
    const long long tokens = (rpp - 1) / a.H + 2;
    return vec && tokens * (a.r / 2) <= NR_PAIRS && passes(a.M * a.H, a.d, 4) >= 256 ? 4 : 1;
}
int norm_rope_blocks(long long rows, int d) {
    const long long p = passes(rows, d, 1);
    return p < 1024 ? (int)p : 1024;
}

template <bool BF> static hipError_t norm_launch(const NormRopeArgs &a, bool back, unsigned grid, hipStream_t st) {
    const int lpr = lanes_per_row(a.d);
    const bool vec = row_vectors(a.d, a.r, a.inter);
    const dim3 g(grid), t(NR_THREADS);
    if (vec && rows_per_thread(a, vec) == 4) {
        if (back) hipLaunchKernelGGL((norm_rope_bwd_kernel<BF, true, 4>), g, t, 0, st, a, lpr);
        else hipLaunchKernelGGL((norm_rope_kernel<BF, true, 4>), g, t, 0, st, a, lpr);
    } else if (vec) {
        if (back) hipLaunchKernelGGL((norm_rope_bwd_kernel<BF, true, 1>), g, t, 0, st, a, lpr);
        else hipLaunchKernelGGL((norm_rope_kernel<BF, true, 1>), g, t, 0, st, a, lpr);
    } else {
        if (back) hipLaunchKernelGGL((norm_rope_bwd_kernel<BF, false, 1>), g, t, 0, st, a, lpr);
        else hipLaunchKernelGGL((norm_rope_kernel<BF, false, 1>), g, t, 0, st, a, lpr);
    }
    return hipGetLastError();
}
hipError_t launch_norm_rope(const NormRopeArgs &a, bool bf16, hipStream_t st) {
    const long long p = passes(a.M * a.H, a.d, rows_per_thread(a, row_vectors(a.d, a.r, a.inter)));
    const unsigned grid = (unsigned)(p < 16384 ? p : 16384);
    return bf16 ? norm_launch<true>(a, false, grid, st) : norm_launch<false>(a, false, grid, st);
}
hipError_t launch_norm_rope_bwd(const NormRopeArgs &a, bool bf16, hipStream_t st) {
    return bf16 ? norm_launch<true>(a, true, (unsigned)a.nblk, st) : norm_launch<false>(a, true, (unsigned)a.nblk, st);
}
hipError_t launch_norm_sum(const NormRopeArgs &a, hipStream_t st) {
    hipLaunchKernelGGL(norm_sum_kernel, dim3((unsigned)((a.d + 3) / 4)), dim3(256), 0, st, a);
    return hipGetLastError();
}

// A new token's cache row: its latent normalised, its rotary key turned, at
// the slot the plan gave it. A group of LPR lanes takes the latents of UN
// tokens, requested together; the pairs of the workgroup's tokens are shared
// by all its threads (each pair's turn is needed once, so it is formed where
// it is used). Slots outside the pool (-1: none) are skipped. Bound by the
// rows' bytes (32768 rows of 512 + 64 bf16: 20 us, 3.9 TB/s; 256 rows: 4 us,
// the launch).
template <bool BF, int UN> __global__ __launch_bounds__(NR_THREADS) void mla_write_kernel(MlaWriteArgs a, int lpr) {
    using S = typename Op<BF>::S;
    const int slots = NR_THREADS / lpr, sub = threadIdx.x % lpr, d = a.dl + a.dr, hp = a.dr / 2;
    const int i0 = blockIdx.x * slots * UN, first = i0 + threadIdx.x / lpr;
    Raw<BF, true> c[UN];
    int slot[UN];
#pragma unroll
    for (int u = 0; u < UN; ++u) {
        const int i = first + u * slots;
        slot[u] = i < a.n ? a.slots[i] : -1;
        if (slot[u] >= a.n_slots) slot[u] = -1;
        c[u].load((const S *)a.c + (size_t)(i < a.n ? i : 0) * a.dl, sub, lpr, a.dl, i < a.n);
    }
    for (int e = threadIdx.x; e < slots * UN * hp; e += NR_THREADS) {
        const int i = i0 + e / hp;
        if (i >= a.n) break;
        const int at = a.slots[i], p = e % hp;
        const int ca = a.inter ? 2 * p : p, cb = a.inter ? 2 * p + 1 : p + hp;
        const S *kr = (const S *)a.kr + (size_t)i * a.dr;
        S ka = kr[ca], kb = kr[cb];
        if (a.freqs) { // (else as they are: a turn by no angle would make inf * 0 of a partner)
            const float x = to_f(ka), y = to_f(kb);
            const float2 t = turn_of(a.pos[i], a.freqs[p]);
            ka = from_f<BF>(x * t.x - y * t.y);
            kb = from_f<BF>(y * t.x + x * t.y);
        }
        if (at < 0 || at >= a.n_slots) continue;
        S *row = (S *)a.cache + (size_t)at * d + a.dl;
        row[ca] = ka;
        row[cb] = kb;
    }
    float w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = a.w && sub * 8 < a.dl ? a.w[sub * 8 + j] : 1.f;
#pragma unroll
    for (int u = 0; u < UN; ++u) {
        float v[8];
        c[u].values(v);
        float inv = 1.f;
        if (a.norm) {
            float ss = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(v[j], v[j], ss);
            inv = rsqrtf(fmaf(lanes_sum(ss, lpr), 1.f / (float)a.dl, a.eps));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= inv * w[j];
        if (slot[u] >= 0) store_row<BF, true>((S *)a.cache + (size_t)slot[u] * d, sub, lpr, a.dl, v);
    }
}

template <bool BF> static void write_launch(const MlaWriteArgs &a, hipStream_t st) {
    const int lpr = lanes_per_row(a.dl);
    const long long per = NR_THREADS / lpr;
    // four tokens per lane group once that leaves a workgroup for every CU
    if ((a.n + 4 * per - 1) / (4 * per) >= 256)
        hipLaunchKernelGGL((mla_write_kernel<BF, 4>), dim3((unsigned)((a.n + 4 * per - 1) / (4 * per))),
                           dim3(NR_THREADS), 0, st, a, lpr);
    else
        hipLaunchKernelGGL((mla_write_kernel<BF, 1>), dim3((unsigned)((a.n + per - 1) / per)), dim3(NR_THREADS), 0, st,
                           a, lpr);
}
hipError_t launch_mla_write(const MlaWriteArgs &a, bool bf16, hipStream_t st) {
    if (bf16) write_launch<true>(a, st);
    else write_launch<false>(a, st);
    return hipGetLastError();
}

} // namespace gdn
