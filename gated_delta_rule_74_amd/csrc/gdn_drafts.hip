// Drafted tokens against the target's distributions.
//
//   p_i = softmax(z_i / T), q_i likewise; draft x is accepted while u_i q_i(x) < p_i(x);
//   at the first that is not, a token from max(p_i - q_i, 0), else from the next row's p:
//   the lowest v whose running sum passes u_S times the whole sum.
//
// The result is whole numbers that hang on comparisons of long sums, so those
// run in fp64: every exponential to 2^-45 by a polynomial of degree 9, fifteen
// vector instructions in all (the fp64 rate of this chip is that of fp32), where fp32
// exponentials would leave the drawn token open to about V 2^-24. Three launches:
//   sums  every row is cut into pieces that a workgroup holds in registers; a
//         piece's largest logit, and the sum of its exponentials relative to that
//   left  decides, from those sums, how many drafts are accepted (each workgroup
//         of a sequence for itself: a few hundred numbers); where one was
//         rejected, the sums over the same pieces of what is left to draw from
//   draw  finds the piece the drawn token lies in, and the token in it
// The first reads every logit once and is what takes the time.
#include "gdn_common.hpp"
#include "gdn_serve.hpp"

namespace gdn {

constexpr int VT = 256, VPER = 32, VPIECE = VT * VPER; // threads; logits of a thread; of a piece

int verify_pieces(int V, bool) { return (V + VPIECE - 1) / VPIECE; }

// 2^t for t <= 0 (or NaN, which gives 0), to 2^-45: t = k + f with |f| <= 1/2, and
// 2^f by the polynomial that meets it at the ten Chebyshev points of that interval.
__device__ __forceinline__ double exp2_f64(double t) {
    t = fmax(t, -1100.0);
    const double big = 6755399441055744.0, k = t + big; // 1.5 * 2^52: the low bits hold the rounded t
    const double f = t - (k - big);
    double p = 1.0205905320493103e-07;
    p = fma(p, f, 1.3259645243929057e-06);
    p = fma(p, f, 1.5252672925346873e-05);
    p = fma(p, f, 0.00015403433751254997);
    p = fma(p, f, 0.0013333558200793719);
    p = fma(p, f, 0.009618129193934304);
    p = fma(p, f, 0.05550410866465168);
    p = fma(p, f, 0.2402265069564034);
    p = fma(p, f, 0.6931471805599462);
    p = fma(p, f, 1.0000000000000135);
    return __builtin_amdgcn_ldexp(p, (int)(uint32_t)__builtin_bit_cast(uint64_t, k));
}

// sum over a workgroup of VT threads, every thread gets it
__device__ __forceinline__ double block_sum(double x, double *w) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o, 64);
    __syncthreads(); // (the last sum's readers are done)
    if ((threadIdx.x & 63) == 0) w[threadIdx.x >> 6] = x;
    __syncthreads();
    return (w[0] + w[1]) + (w[2] + w[3]);
}

// maximum that a NaN survives
__device__ __forceinline__ float max_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// Logits of a row: a group of eight (four) that covers the places from i on.
// Rows begin anywhere; the last group of a row is read from further left, so that
// nothing outside the row is read, and -inf stands for the places before i then.
// Returns the place of z[0].
template <bool BF> struct Logits {
    using S = typename Op<BF>::S;
    static constexpr int G = Op<BF>::VEC; // logits of a 16-byte group
    struct __attribute__((packed, aligned(sizeof(S)))) Group {
        S x[G];
    };
    static __device__ __forceinline__ int get(const S *row, int V, int i, float (&z)[G]) {
        if (V < G) { // (shorter than a group)
#pragma unroll
            for (int e = 0; e < G; ++e) z[e] = i + e < V ? to_f(row[min(i + e, V - 1)]) : -INFINITY;
            return i;
        }
        const int at = min(i, V - G), skip = i - at; // skip > 0: the row's end
        const Group w = *(const Group *)(row + at);
#pragma unroll
        for (int e = 0; e < G; ++e) z[e] = to_f(w.x[e]);
        if (skip > 0) {
#pragma unroll
            for (int e = 0; e < G; ++e) z[e] = e >= skip ? z[e] : -INFINITY;
        }
        return at;
    }
};

__device__ __forceinline__ int drafts_of(const VerifyArgs &a, int n) {
    return a.dlens ? min(max(a.dlens[n], 0), a.S) : a.S;
}
__device__ __forceinline__ float heat_of(const VerifyArgs &a, int n) { return a.temp ? a.temp[n] : 1.f; }
// scale of a logit in powers of two
__device__ __forceinline__ double unit_of(float heat) { return heat > 0.f ? LOG2E / (double)heat : LOG2E; }

template <bool BF> __global__ __launch_bounds__(VT) void verify_sums_kernel(VerifyArgs a) {
    using S = typename Op<BF>::S;
    constexpr int G = Op<BF>::VEC, NG = VPER / G;
    __shared__ double ws[4];
    __shared__ float wm[4];
    __shared__ int wi[4];
    const int tid = threadIdx.x, target = a.N * (a.S + 1);
    const int row = blockIdx.x / a.nch, piece = blockIdx.x % a.nch;
    // rows that no draft reaches are not read, nor greedy sequences' drafts
    const int n = row < target ? row / (a.S + 1) : (row - target) / a.S;
    const float heat = heat_of(a, n);
    const bool greedy = !(heat > 0.f);
    if (row < target ? row % (a.S + 1) > drafts_of(a, n) : greedy || (row - target) % a.S >= drafts_of(a, n)) return;
    const S *z0 = row < target ? (const S *)a.logits + (size_t)row * a.V : (const S *)a.dlogits + (size_t)(row - target) * a.V;
    float z[NG][G];
    int at[NG];
#pragma unroll
    for (int k = 0; k < NG; ++k) at[k] = Logits<BF>::get(z0, a.V, piece * VPIECE + (k * VT + tid) * G, z[k]);
    float m = z[0][0];
#pragma unroll
    for (int k = 0; k < NG; ++k)
#pragma unroll
        for (int e = 0; e < G; ++e) m = max_nan(m, z[k][e]);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = max_nan(m, __shfl_xor(m, o, 64));
    if ((tid & 63) == 0) wm[tid >> 6] = m;
    __syncthreads();
    m = max_nan(max_nan(wm[0], wm[1]), max_nan(wm[2], wm[3]));
    double sum = 0.0;
    if (m > -INFINITY && m < INFINITY) {
        const double c = unit_of(heat), top = m; // (their difference is exact, however small a temperature divides it)
#pragma unroll
        for (int k = 0; k < NG; ++k)
#pragma unroll
            for (int e = 0; e < G; ++e) sum += exp2_f64(((double)z[k][e] - top) * c);
    }
    sum = block_sum(sum, ws);
    if (greedy) { // first place of the largest
        int best = 2147483647;
#pragma unroll
        for (int k = NG - 1; k >= 0; --k)
#pragma unroll
            for (int e = G - 1; e >= 0; --e)
                if (z[k][e] == m) best = at[k] + e;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) best = min(best, __shfl_xor(best, o, 64));
        if ((tid & 63) == 0) wi[tid >> 6] = best;
        __syncthreads();
        if (tid == 0) a.best[blockIdx.x] = min(min(wi[0], wi[1]), min(wi[2], wi[3]));
    }
    if (tid == 0) {
        a.sums[blockIdx.x] = sum;
        a.tops[blockIdx.x] = m;
    }
}

// A row's distribution: log2 p(v) = (z_v - top) c - sum; sum NaN: it has none.
struct Dist {
    double top, sum; // largest logit; log2 of the sum of the exponentials relative to it
};
__device__ __forceinline__ double log2_p(double z, const Dist &d, double c) { return (z - d.top) * c - d.sum; }
// from its pieces' sums, by one wave
__device__ __forceinline__ Dist row_dist(const VerifyArgs &a, int row, double c, int lane) {
    const size_t at = (size_t)row * a.nch;
    float m = -INFINITY;
    for (int i = lane; i < a.nch; i += 64) m = max_nan(m, a.tops[at + i]);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = max_nan(m, __shfl_xor(m, o, 64));
    double s = 0.0;
    if (m > -INFINITY && m < INFINITY)
        for (int i = lane; i < a.nch; i += 64) {
            const float t = a.tops[at + i];
            if (t > -INFINITY) s += a.sums[at + i] * exp2_f64(((double)t - (double)m) * c);
        }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
    return {(double)m, s > 0.0 ? log2(s) : __builtin_nan("")};
}
// first largest place of a row, by one wave
__device__ __forceinline__ int row_best(const VerifyArgs &a, int row, double top, int lane) {
    const size_t at = (size_t)row * a.nch;
    int best = 2147483647;
    for (int i = lane; i < a.nch; i += 64)
        if ((double)a.tops[at + i] == top) best = min(best, a.best[at + i]);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) best = min(best, __shfl_xor(best, o, 64));
    return best;
}
template <bool BF> __device__ __forceinline__ double logit_at(const void *z, size_t row, int V, int v) {
    return (double)to_f(((const typename Op<BF>::S *)z)[row * V + v]);
}
__device__ __forceinline__ double uniform_of(float u) { // in [0, 1)
    return (double)fminf(u > 0.f ? u : 0.f, 0.99999994f);
}

// What was decided for a sequence, in VerifyArgs::pick.
enum { PICK_ROW = 0, PICK_MODE, PICK_TOKEN, PICK_P, PICK_Q = PICK_P + 2 }; // (P, Q: top and sum)
enum { MODE_NONE = 0, MODE_TOKEN, MODE_ROW, MODE_DIFF, MODE_WITHOUT }; // nothing; known; p; p - q; p without the draft

// Decides sequence n: by one workgroup, each wave every fourth row.
struct Choice {
    int row, mode, token;
    Dist p, q;
};
template <bool BF> __device__ __forceinline__ Choice decide(const VerifyArgs &a, int n, Choice *rows, bool write) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, L = drafts_of(a, n);
    const float heat = heat_of(a, n);
    const bool greedy = !(heat > 0.f);
    const double c = unit_of(heat);
    __shared__ int stop;
    if (tid == 0) stop = L;
    __syncthreads();
    // rows in order, four at a time, until one stops
    Choice mine = {};
    for (int i0 = 0; i0 <= L; i0 += 4) {
        const int i = i0 + wave;
        if (i <= L) {
            const int row = n * (a.S + 1) + i;
            const Dist p = row_dist(a, row, c, lane);
            const bool none = !(p.sum == p.sum);
            const int x = i < L ? a.draft[(size_t)n * a.S + i] : -1;
            const bool inside = (unsigned)x < (unsigned)a.V;
            mine = {i, MODE_ROW, -1, p, p};
            bool yes = false;
            if (none) {
                mine.mode = MODE_NONE;
            } else if (greedy) {
                mine.mode = MODE_TOKEN;
                mine.token = row_best(a, row, p.top, lane);
                yes = i < L && x == mine.token;
            } else if (i < L && inside) {
                const double lp = log2_p(logit_at<BF>(a.logits, row, a.V, x), p, c);
                double lq = 0.0;
                bool known = true;
                mine.mode = MODE_WITHOUT;
                if (a.dlogits) {
                    const Dist q = row_dist(a, a.N * (a.S + 1) + n * a.S + i, c, lane);
                    known = q.sum == q.sum;
                    mine.mode = known ? MODE_DIFF : MODE_ROW;
                    mine.q = q;
                    lq = log2_p(logit_at<BF>(a.dlogits, (size_t)n * a.S + i, a.V, x), q, c);
                }
                yes = known && uniform_of(a.uniforms[(size_t)n * (a.S + 1) + i]) * exp2(lq) < exp2(lp);
            }
            if (lane == 0) {
                if (!yes) atomicMin(&stop, i);
                if (yes && write) {
                    a.tokens[(size_t)n * (a.S + 1) + i] = x;
                    if (a.logprobs)
                        a.logprobs[(size_t)n * (a.S + 1) + i] =
                            (float)(log2_p(logit_at<BF>(a.logits, row, a.V, x), p, c) / LOG2E);
                }
            }
        }
        __syncthreads();
        if (stop < i0 + 4) break; // (uniform)
    }
    if (lane == 0 && mine.row == stop && wave == (stop & 3)) *rows = mine;
    __syncthreads();
    return *rows;
}

// p(v), or what is left of it, at a place of the row.
__device__ __forceinline__ double left_of(int mode, float zp, float zq, double c, const Dist &dp, const Dist &dq, int v, int x) {
    const double p = exp2_f64(log2_p((double)zp, dp, c));
    if (mode == MODE_DIFF) return fmax(p - exp2_f64(log2_p((double)zq, dq, c)), 0.0);
    return mode == MODE_WITHOUT && v == x ? 0.0 : p;
}

template <bool BF> __global__ __launch_bounds__(VT) void verify_left_kernel(VerifyArgs a) {
    using S = typename Op<BF>::S;
    constexpr int G = Op<BF>::VEC, NG = VPER / G;
    __shared__ double ws[4];
    __shared__ Choice shared;
    const int n = blockIdx.x / a.nch, piece = blockIdx.x % a.nch, tid = threadIdx.x;
    const Choice d = decide<BF>(a, n, &shared, piece == 0);
    if (piece == 0) {
        if (tid == 0) {
            a.accepted[n] = d.row;
            double *pick = a.pick + (size_t)n * VERIFY_PICK;
            pick[PICK_ROW] = d.row;
            pick[PICK_MODE] = d.mode;
            pick[PICK_TOKEN] = d.token;
            pick[PICK_P] = d.p.top;
            pick[PICK_P + 1] = d.p.sum;
            pick[PICK_Q] = d.q.top;
            pick[PICK_Q + 1] = d.q.sum;
        }
        for (int i = d.row + 1 + tid; i <= a.S; i += VT) {
            a.tokens[(size_t)n * (a.S + 1) + i] = -1;
            if (a.logprobs) a.logprobs[(size_t)n * (a.S + 1) + i] = 0.f;
        }
    }
    if (d.mode != MODE_DIFF && d.mode != MODE_WITHOUT) return;
    const double c = unit_of(heat_of(a, n));
    const int x = a.draft[(size_t)n * a.S + d.row];
    const S *zp = (const S *)a.logits + ((size_t)n * (a.S + 1) + d.row) * a.V;
    const S *zq = d.mode == MODE_DIFF ? (const S *)a.dlogits + ((size_t)n * a.S + d.row) * a.V : zp;
    float p[NG][G], q[NG][G];
    int at[NG];
#pragma unroll
    for (int k = 0; k < NG; ++k) {
        at[k] = Logits<BF>::get(zp, a.V, piece * VPIECE + (k * VT + tid) * G, p[k]);
        Logits<BF>::get(zq, a.V, piece * VPIECE + (k * VT + tid) * G, q[k]);
    }
    double sum = 0.0;
#pragma unroll
    for (int k = 0; k < NG; ++k)
#pragma unroll
        for (int e = 0; e < G; ++e)
            sum += left_of(d.mode, p[k][e], q[k][e], c, d.p, d.q, at[k] + e, x);
    sum = block_sum(sum, ws);
    if (tid == 0) a.left[blockIdx.x] = sum;
}

template <bool BF> __global__ __launch_bounds__(VT) void verify_draw_kernel(VerifyArgs a) {
    using S = typename Op<BF>::S;
    constexpr int G = Op<BF>::VEC, NG = VPER / G;
    __shared__ double ends[VT];
    __shared__ int found, where;
    __shared__ double rest;
    const int n = blockIdx.x, tid = threadIdx.x;
    const double *pick = a.pick + (size_t)n * VERIFY_PICK;
    const int i = (int)pick[PICK_ROW], mode = (int)pick[PICK_MODE];
    const size_t out = (size_t)n * (a.S + 1) + i;
    const double c = unit_of(heat_of(a, n));
    const Dist dp = {pick[PICK_P], pick[PICK_P + 1]}, dq = {pick[PICK_Q], pick[PICK_Q + 1]};
    auto emit = [&](int v) {
        a.tokens[out] = v;
        if (a.logprobs)
            a.logprobs[out] = v < 0 ? 0.f : (float)(log2_p(logit_at<BF>(a.logits, out, a.V, v), dp, c) / LOG2E);
    };
    if (mode == MODE_NONE || mode == MODE_TOKEN) {
        if (tid == 0) emit(mode == MODE_TOKEN ? (int)pick[PICK_TOKEN] : -1);
        return;
    }
    // the piece: the first whose end passes u times the whole (should none, the last with anything), by one wave
    if (tid < 64) {
        const size_t at = (mode == MODE_ROW ? out : (size_t)n) * a.nch;
        auto part = [&](int k) {
            if (k >= a.nch) return 0.0;
            if (mode != MODE_ROW) return a.left[at + k];
            return a.tops[at + k] > -INFINITY ? a.sums[at + k] * exp2(log2_p((double)a.tops[at + k], dp, c)) : 0.0;
        };
        double all = 0.0;
        for (int k = tid; k < a.nch; k += 64) all += part(k);
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) all += __shfl_xor(all, o, 64);
        const double aim = uniform_of(a.uniforms[(size_t)n * (a.S + 1) + a.S]) * all;
        double before = 0.0, start = 0.0;
        int piece = -1;
        for (int k0 = 0; k0 < a.nch; k0 += 64) {
            const double own = part(k0 + tid);
            double s = own;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const double y = __shfl_up(s, o, 64);
                if (tid >= o) s += y;
            }
            const uint64_t some = __ballot(own > 0.0), past = __ballot(own > 0.0 && before + s > aim);
            if (some) {
                const int l = past ? __builtin_ctzll(past) : 63 - __builtin_clzll(some);
                piece = k0 + l;
                start = before + __shfl(s - own, l, 64);
            }
            if (past) break;
            before += __shfl(s, 63, 64);
        }
        if (tid == 0) {
            where = piece;
            rest = aim - start; // to be passed within the piece
            found = 2147483647;
        }
    }
    __syncthreads();
    const int piece = where;
    if (piece < 0) { // (nothing left: not with finite numbers)
        if (tid == 0) emit(-1);
        return;
    }
    const int x = mode == MODE_ROW ? -1 : a.draft[(size_t)n * a.S + i];
    const S *zp = (const S *)a.logits + out * a.V;
    const S *zq = mode == MODE_DIFF ? (const S *)a.dlogits + ((size_t)n * a.S + i) * a.V : zp;
    // places in order: a thread takes VPER in a row
    const int v0 = piece * VPIECE + tid * VPER;
    double r[NG][G], mine = 0.0;
    int place[NG];
#pragma unroll
    for (int k = 0; k < NG; ++k) {
        float p[G], q[G];
        place[k] = Logits<BF>::get(zp, a.V, v0 + k * G, p);
        Logits<BF>::get(zq, a.V, v0 + k * G, q);
#pragma unroll
        for (int e = 0; e < G; ++e) {
            r[k][e] = left_of(mode, p[e], q[e], c, dp, dq, place[k] + e, x);
            mine += r[k][e];
        }
    }
    ends[tid] = mine;
    __syncthreads();
    for (int o = 1; o < VT; o <<= 1) {
        const double y = tid >= o ? ends[tid - o] : 0.0;
        __syncthreads();
        ends[tid] += y;
        __syncthreads();
    }
    // the first place whose running sum passes `rest`; should rounding leave none, the last with anything
    double s = tid ? ends[tid - 1] : 0.0;
    int hit = 2147483647, last = -1;
#pragma unroll
    for (int k = 0; k < NG; ++k)
#pragma unroll
        for (int e = 0; e < G; ++e) {
            s += r[k][e];
            const int v = place[k] + e;
            if (r[k][e] > 0.0) {
                last = v;
                if (s > rest) hit = min(hit, v);
            }
        }
    if (tid == 0) where = -1;
    __syncthreads();
    atomicMin(&found, hit);
    atomicMax(&where, last);
    __syncthreads();
    if (tid == 0) emit(found != 2147483647 ? found : where);
}

hipError_t launch_verify_sums(const VerifyArgs &a, bool bf16, hipStream_t st) {
    const long long rows = (long long)a.N * (a.S + 1) + (a.dlogits ? (long long)a.N * a.S : 0);
    const dim3 grid((unsigned)(rows * a.nch));
    if (bf16) hipLaunchKernelGGL(verify_sums_kernel<true>, grid, dim3(VT), 0, st, a);
    else hipLaunchKernelGGL(verify_sums_kernel<false>, grid, dim3(VT), 0, st, a);
    return hipGetLastError();
}
hipError_t launch_verify_left(const VerifyArgs &a, bool bf16, hipStream_t st) {
    const dim3 grid((unsigned)((long long)a.N * a.nch));
    if (bf16) hipLaunchKernelGGL(verify_left_kernel<true>, grid, dim3(VT), 0, st, a);
    else hipLaunchKernelGGL(verify_left_kernel<false>, grid, dim3(VT), 0, st, a);
    return hipGetLastError();
}
hipError_t launch_verify_draw(const VerifyArgs &a, bool bf16, hipStream_t st) {
    if (bf16) hipLaunchKernelGGL(verify_draw_kernel<true>, dim3(a.N), dim3(VT), 0, st, a);
    else hipLaunchKernelGGL(verify_draw_kernel<false>, dim3(a.N), dim3(VT), 0, st, a);
    return hipGetLastError();
}

} // namespace gdn
