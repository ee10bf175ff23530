// Drafted tokens against the target's distributions.
//
//   p_i = softmax(z_i / T), q_i likewise; draft x is accepted while u_i q_i(x) < p_i(x);
//   at the first that is not, a token from max(p_i - q_i, 0), else from the next row's p:
//   the lowest v whose running sum passes u_S times the whole sum.
//
// The result is whole numbers that hang on comparisons of long sums, so those
// run in fp64 (the chip's fp64 rate is that of fp32): fp32 exponentials would
// leave the drawn token open to about V 2^-24. Four launches:
//   sums    every row is cut into pieces; a piece's sum of exponentials, and its
//           largest logit. Reads every logit once and takes most of the time.
//   decide  from those, how many drafts are accepted, and what is to be drawn from
//   left    where that is what a rejected draft leaves, max(p - q, 0): its sums over
//           the same pieces
//   draw    finds the piece the drawn token lies in, the thread, and the token
// 256 sequences of two drafts, V 65792, bf16: 43, 6, 23 and 10 us; the sums by the exponentials' fp64
// instructions (59 % of the vector units' time, 93 MB of logits), the rest by the chains of
// loads and sums that follow one another. Three sequences of four, V 32001, fp32: 5, 4, 4 and 9.
// A piece is a wave's, which needs no other for it. Its loop is kept rolled:
// unrolled over all of a lane's logits the code is tens of KB that every launch
// fetches anew (256 sequences, V 65792: 50 us for the sums, 33 for what is left).
#include "gdn_common.hpp"
#include "gdn_serve.hpp"

namespace gdn {

constexpr int VPIECE = 2048;    // logits of a piece
constexpr int VT = 256, DT = 256; // threads of the workgroups, and of those of draw

int verify_pieces(int V) { return (V + VPIECE - 1) / VPIECE; }

// 2^t for t up to 1000 (below -1100, or NaN: 0): t = k + f with |f| <= 1/2, and 2^f by
// the polynomial that meets it at the Chebyshev points of that interval. Eight terms,
// 2^-34, for the many logits of a row: a border of the running sum moves by what of that does
// not average out, far less than tokens' borders lie apart. Ten, 2^-45, elsewhere.
template <int TERMS> __device__ __forceinline__ double exp2_part(double f) {
    double p;
    if constexpr (TERMS == 8) {
        p = 1.5303700711232526e-05;
        p = fma(p, f, 0.000154697292141169);
        p = fma(p, f, 0.0013333478473686068);
        p = fma(p, f, 0.009618025613318041);
        p = fma(p, f, 0.05550410906325866);
        p = fma(p, f, 0.24022651213498092);
        p = fma(p, f, 0.6931471805568324);
        p = fma(p, f, 0.9999999999595618);
    } else {
        p = 1.0205905320493103e-07;
        p = fma(p, f, 1.3259645243929057e-06);
        p = fma(p, f, 1.5252672925346873e-05);
        p = fma(p, f, 0.00015403433751254997);
        p = fma(p, f, 0.0013333558200793719);
        p = fma(p, f, 0.009618129193934304);
        p = fma(p, f, 0.05550410866465168);
        p = fma(p, f, 0.2402265069564034);
        p = fma(p, f, 0.6931471805599462);
        p = fma(p, f, 1.0000000000000135);
    }
    return p;
}
template <int TERMS> __device__ __forceinline__ double exp2_f64(double t) {
    t = fmax(t, -1100.0);
    const double big = 6755399441055744.0, k = t + big; // 1.5 * 2^52: the low bits hold the rounded t
    return __builtin_amdgcn_ldexp(exp2_part<TERMS>(t - (k - big)), __double2loint(k));
}
// The same for -1000 <= t <= 1000 alone, where the factor 2^k is a sum of exponents.
__device__ __forceinline__ double exp2_near(double t) {
    const double big = 6755399441055744.0, k = t + big;
    const double p = exp2_part<8>(t - (k - big));
    return __hiloint2double(__double2hiint(p) + (__double2loint(k) << 20), __double2loint(p));
}

// A row's distribution: log2 p(v) = (z_v - ref) c - sum; sum NaN: it has none. (The difference is exact, however
// small a temperature c divides by.)
struct Dist {
    double ref, sum; // a logit; log2 of the sum of the exponentials relative to it
};
__device__ __forceinline__ double log2_p(double z, const Dist &d, double c) { return fma(z - d.ref, c, -d.sum); }

__device__ __forceinline__ double wave_sum_d(double x) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o, 64);
    return x;
}

// maximum that a NaN survives
__device__ __forceinline__ float max_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// A group of eight (four) logits of a row that covers the places from i on, as
// loaded. Rows begin anywhere; the last group of a row is read from further left,
// so that nothing outside the row is read, and its places before i count as -inf.
template <bool BF> struct Group {
    using S = typename Op<BF>::S;
    static constexpr int G = Op<BF>::VEC;
    struct __attribute__((packed, aligned(sizeof(S)))) Raw {
        S x[G];
    };
    Raw w;
    // place of the first
    static __device__ __forceinline__ int place(int V, int i) { return V < G ? i : min(i, V - G); }
    __device__ __forceinline__ void load(const S *row, int V, int i) {
        if (V < G) { // (shorter than a group)
#pragma unroll
            for (int e = 0; e < G; ++e) w.x[e] = row[min(i + e, V - 1)];
            return;
        }
        w = *(const Raw *)(row + place(V, i));
    }
    // tail: some of the wave's groups may pass the row's end (the same for all lanes, so that others pay nothing)
    __device__ __forceinline__ void get(int V, int i, bool tail, float (&z)[G]) const {
#pragma unroll
        for (int e = 0; e < G; ++e) z[e] = to_f(w.x[e]);
        if (tail) {
            const int from = i - place(V, i), to = V - place(V, i); // those that count
#pragma unroll
            for (int e = 0; e < G; ++e) z[e] = e >= from && e < to ? z[e] : -INFINITY;
        }
    }
};

// f(first place, logits) for a lane's groups of the wave's piece [base, end); two are requested ahead.
template <bool BF, class F>
__device__ __forceinline__ void each_group(const typename Op<BF>::S *row, int V, int base, int end, int lane, F &&f) {
    constexpr int G = Op<BF>::VEC, STEP = 64 * G;
    const int mine = lane * G;
    Group<BF> a, b;
    a.load(row, V, base + mine);
    if (base + STEP < end) b.load(row, V, base + STEP + mine);
#pragma unroll 1
    for (int i = base; i < end; i += STEP) {
        float z[G];
        a.get(V, i + mine, i + STEP > V, z);
        a = b;
        if (i + 2 * STEP < end) b.load(row, V, i + 2 * STEP + mine);
        f(Group<BF>::place(V, i + mine), z);
    }
}

__device__ __forceinline__ int drafts_of(const VerifyArgs &a, int n) {
    return a.dlens ? min(max(a.dlens[n], 0), a.S) : a.S;
}
__device__ __forceinline__ float heat_of(const VerifyArgs &a, int n) { return a.temp ? a.temp[n] : 1.f; }
// scale of a logit in powers of two
__device__ __forceinline__ double unit_of(float heat) { return heat > 0.f ? LOG2E / (double)heat : LOG2E; }

template <bool BF> __global__ __launch_bounds__(VT) void verify_sums_kernel(VerifyArgs a) {
    using S = typename Op<BF>::S;
    constexpr int G = Op<BF>::VEC;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), target = a.N * (a.S + 1);
    const int row = blockIdx.x, piece = blockIdx.y * (VT / 64) + wave, base = piece * VPIECE, end = min(base + VPIECE, a.V);
    // rows that no draft reaches are not read, nor greedy sequences' drafts
    const int n = row < target ? row / (a.S + 1) : (row - target) / a.S;
    const int i = row < target ? row - n * (a.S + 1) : row - target - n * a.S;
    const float heat = heat_of(a, n);
    const bool greedy = !(heat > 0.f);
    if (piece >= a.nch || (row < target ? i > drafts_of(a, n) : greedy || i >= drafts_of(a, n))) return;
    const S *z0 = row < target ? (const S *)a.logits + (size_t)row * a.V : (const S *)a.dlogits + (size_t)(row - target) * a.V;
    // One pass: fp64 holds the exponentials of usual logits as they are, relative to a logit of 0.
    const double c = unit_of(heat);
    float m = -INFINITY;
    double sum = 0.0;
    each_group<BF>(z0, a.V, base, end, lane, [&](int, const float(&z)[G]) {
#pragma unroll
        for (int e = 0; e < G; ++e) {
            m = max_nan(m, z[e]);
            sum += exp2_near(fmax((double)z[e] * c, -1000.0));
        }
    });
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = max_nan(m, __shfl_xor(m, o, 64));
    float ref = 0.f;
    if (!(fabs((double)m * c) < 900.0)) { // else relative to the largest, in a second one
        ref = m;
        sum = 0.0;
        if (m > -INFINITY && m < INFINITY)
            each_group<BF>(z0, a.V, base, end, lane, [&](int, const float(&z)[G]) {
#pragma unroll
                for (int e = 0; e < G; ++e) sum += exp2_near(fmax(((double)z[e] - (double)m) * c, -1000.0));
            });
    }
    sum = wave_sum_d(sum);
    const size_t out = (size_t)row * a.nch + piece;
    if (greedy) { // first place of the largest
        int best = 2147483647;
        each_group<BF>(z0, a.V, base, end, lane, [&](int at, const float(&z)[G]) {
#pragma unroll
            for (int e = 0; e < G; ++e)
                if (z[e] == m) best = min(best, at + e);
        });
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) best = min(best, __shfl_xor(best, o, 64));
        if (lane == 0) a.best[out] = best;
    }
    if (lane == 0) {
        a.sums[out] = sum;
        a.tops[out] = m;
        a.refs[out] = ref;
    }
}

// A row's distribution and its largest logit, from its pieces' sums, by one wave. (A piece of -inf alone has
// -inf for its reference, and no sum.)
__device__ __forceinline__ Dist row_dist(const VerifyArgs &a, int row, double c, int lane, float &top) {
    const size_t at = (size_t)row * a.nch;
    float m = -INFINITY, ref = -INFINITY;
    for (int i = lane; i < a.nch; i += 64) {
        m = max_nan(m, a.tops[at + i]);
        ref = fmaxf(ref, a.refs[at + i]);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        m = max_nan(m, __shfl_xor(m, o, 64));
        ref = fmaxf(ref, __shfl_xor(ref, o, 64));
    }
    top = m;
    double s = 0.0;
    if (m > -INFINITY && m < INFINITY)
        for (int i = lane; i < a.nch; i += 64) {
            const float r = a.refs[at + i];
            if (r > -INFINITY) s += a.sums[at + i] * exp2_f64<10>(((double)r - (double)ref) * c);
        }
    s = wave_sum_d(s);
    return {(double)ref, s > 0.0 ? log2(s) : __builtin_nan("")};
}
// first largest place of a row, by one wave
__device__ __forceinline__ int row_best(const VerifyArgs &a, int row, float top, int lane) {
    const size_t at = (size_t)row * a.nch;
    int best = 2147483647;
    for (int i = lane; i < a.nch; i += 64)
        if (a.tops[at + i] == top) best = min(best, a.best[at + i]);
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
enum { PICK_ROW = 0, PICK_MODE, PICK_P, PICK_Q = PICK_P + 2, PICK_UNIT = PICK_Q + 2 };
enum { MODE_NONE = 0, MODE_TOKEN, MODE_ROW, MODE_DIFF, MODE_WITHOUT }; // nothing; known; p; p - q; p without the draft

// Decides a sequence, one workgroup, each wave every fourth row.
struct Choice {
    int row, mode, token;
    Dist p, q;
};
template <bool BF> __global__ __launch_bounds__(VT) void verify_decide_kernel(VerifyArgs a) {
    __shared__ int stop;
    const int n = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, L = drafts_of(a, n);
    const float heat = heat_of(a, n);
    const bool greedy = !(heat > 0.f);
    const double c = unit_of(heat);
    if (tid == 0) stop = L;
    __syncthreads();
    // rows in order, four at a time, until one stops
    Choice mine = {};
    for (int i0 = 0; i0 <= L; i0 += 4) {
        const int i = i0 + wave;
        if (i <= L) {
            const int row = n * (a.S + 1) + i, drow = n * a.S + i;
            const bool sampled = !greedy && i < L;
            const int x = i < L ? a.draft[drow] : -1;
            const bool inside = (unsigned)x < (unsigned)a.V;
            // (requested before the sums are added up)
            const double zp = logit_at<BF>(a.logits, row, a.V, inside ? x : 0);
            const double zq = sampled && a.dlogits ? logit_at<BF>(a.dlogits, drow, a.V, inside ? x : 0) : 0.0;
            const float u = a.uniforms[row];
            float top, qtop;
            const Dist p = row_dist(a, row, c, lane, top);
            mine = {i, MODE_ROW, -1, p, p};
            bool yes = false;
            if (!(p.sum == p.sum)) {
                mine.mode = MODE_NONE;
            } else if (greedy) {
                mine.mode = MODE_TOKEN;
                mine.token = row_best(a, row, top, lane);
                yes = i < L && x == mine.token;
            } else if (i < L && inside) {
                double lq = 0.0;
                bool known = true;
                mine.mode = MODE_WITHOUT;
                if (a.dlogits) {
                    mine.q = row_dist(a, a.N * (a.S + 1) + drow, c, lane, qtop);
                    known = mine.q.sum == mine.q.sum;
                    mine.mode = known ? MODE_DIFF : MODE_ROW;
                    lq = log2_p(zq, mine.q, c);
                }
                yes = known && uniform_of(u) * exp2_f64<10>(lq) < exp2_f64<10>(log2_p(zp, p, c));
            }
            if (lane == 0) {
                if (!yes) atomicMin(&stop, i);
                if (yes) {
                    a.tokens[row] = x;
                    if (a.logprobs) a.logprobs[row] = (float)(log2_p(zp, p, c) / LOG2E);
                }
            }
        }
        __syncthreads();
        if (stop < i0 + 4) break; // (uniform)
    }
    const int at = stop;
    if (lane == 0 && mine.row == at && wave == (at & 3)) {
        a.accepted[n] = at;
        double *pick = a.pick + (size_t)n * VERIFY_PICK;
        pick[PICK_ROW] = at;
        pick[PICK_MODE] = mine.mode;
        pick[PICK_P] = mine.p.ref;
        pick[PICK_P + 1] = mine.p.sum;
        pick[PICK_Q] = mine.q.ref;
        pick[PICK_Q + 1] = mine.q.sum;
        pick[PICK_UNIT] = c;
        if (mine.mode == MODE_NONE || mine.mode == MODE_TOKEN) { // known already
            const size_t out = (size_t)n * (a.S + 1) + at;
            a.tokens[out] = mine.token;
            if (a.logprobs)
                a.logprobs[out] =
                    mine.token < 0 ? 0.f : (float)(log2_p(logit_at<BF>(a.logits, out, a.V, mine.token), mine.p, c) / LOG2E);
        }
    }
    // (after the rows behind the rejected one have had their say above)
    for (int i = at + 1 + tid; i <= a.S; i += VT) {
        a.tokens[(size_t)n * (a.S + 1) + i] = -1;
        if (a.logprobs) a.logprobs[(size_t)n * (a.S + 1) + i] = 0.f;
    }
}

// What a sequence draws from.
template <bool BF> struct Source {
    using S = typename Op<BF>::S;
    static constexpr int G = Op<BF>::VEC;
    int row, mode, x; // x: the rejected draft where there is no more to it, -1: none
    double c;
    Dist p, q;
    const S *zp, *zq;
    __device__ __forceinline__ void whole_row() { // p, whatever was rejected
        mode = MODE_ROW;
        x = -1;
    }
    __device__ __forceinline__ Source(const VerifyArgs &a, int n, int how) : mode(how) {
        const double *pick = a.pick + (size_t)n * VERIFY_PICK;
        row = (int)pick[PICK_ROW];
        p = {pick[PICK_P], pick[PICK_P + 1]};
        q = {pick[PICK_Q], pick[PICK_Q + 1]};
        c = pick[PICK_UNIT];
        x = mode == MODE_WITHOUT ? a.draft[(size_t)n * a.S + row] : -1;
        zp = (const S *)a.logits + ((size_t)n * (a.S + 1) + row) * a.V;
        zq = mode == MODE_DIFF ? (const S *)a.dlogits + ((size_t)n * a.S + row) * a.V : zp;
    }
    __device__ __forceinline__ double weight(float z, float w) const {
        const double r = exp2_f64<8>(log2_p((double)z, p, c));
        return mode == MODE_DIFF ? fmax(r - exp2_f64<8>(log2_p((double)w, q, c)), 0.0) : r;
    }
};

template <bool BF> __global__ __launch_bounds__(VT) void verify_left_kernel(VerifyArgs a) {
    constexpr int G = Op<BF>::VEC, STEP = 64 * G;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // four waves to a piece: there are few of them
    const int n = blockIdx.x, piece = blockIdx.y, base = piece * VPIECE + wave * (VPIECE / 4);
    const int end = min(base + VPIECE / 4, a.V);
    const int mode = (int)a.pick[(size_t)n * VERIFY_PICK + PICK_MODE];
    if (mode != MODE_DIFF && mode != MODE_WITHOUT) return;
    const Source<BF> s(a, n, mode);
    double sum = 0.0;
    if (mode == MODE_WITHOUT) {
        each_group<BF>(s.zp, a.V, base, end, lane, [&](int at, const float(&z)[G]) {
#pragma unroll
            for (int e = 0; e < G; ++e) sum += at + e == s.x ? 0.0 : exp2_f64<8>(log2_p((double)z[e], s.p, s.c));
        });
    } else {
        Group<BF> next; // (the draft's logits)
        next.load(s.zq, a.V, base + lane * G);
        int i = base;
        each_group<BF>(s.zp, a.V, base, end, lane, [&](int, const float(&z)[G]) {
            float w[G];
            next.get(a.V, i + lane * G, i + STEP > a.V, w);
            i += STEP;
            if (i < end) next.load(s.zq, a.V, i + lane * G);
#pragma unroll
            for (int e = 0; e < G; ++e) sum += s.weight(z[e], w[e]);
        });
    }
    __shared__ double ws[4];
    sum = wave_sum_d(sum);
    if (lane == 0) ws[wave] = sum;
    __syncthreads();
    if (threadIdx.x == 0) a.left[(size_t)n * a.nch + piece] = (ws[0] + ws[1]) + (ws[2] + ws[3]);
}

// A rejected draft that leaves less than this (of 1) had the same distribution as the target, as far as the
// exponentials tell: of both their errors, 2^-33 of each probability, no more than 2^-32 can be left.
constexpr double LEFT_LEAST = 0x1p-30;

template <bool BF> __global__ __launch_bounds__(DT) void verify_draw_kernel(VerifyArgs a) {
    constexpr int G = Op<BF>::VEC, PER = VPIECE / DT, NG = PER / G; // places of a thread, in a row
    __shared__ double ws[DT / 64], rest;
    __shared__ int how, where, first, last;
    const int n = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
    const int decided = (int)a.pick[(size_t)n * VERIFY_PICK + PICK_MODE];
    if (decided == MODE_NONE || decided == MODE_TOKEN) return;
    Source<BF> src(a, n, decided);
    const size_t out = (size_t)n * (a.S + 1) + src.row;
    auto emit = [&](int v, float z) {
        a.tokens[out] = v;
        if (a.logprobs) a.logprobs[out] = v < 0 ? 0.f : (float)(log2_p((double)z, src.p, src.c) / LOG2E);
    };
    // the piece: the first whose end passes u times the whole (should none, the last with anything), by one wave
    if (tid < 64) {
        auto part = [&](int k) {
            if (k >= a.nch) return 0.0;
            if (src.mode != MODE_ROW) return a.left[(size_t)n * a.nch + k];
            const size_t at = out * a.nch + k;
            return a.refs[at] > -INFINITY ? a.sums[at] * exp2_f64<10>(log2_p((double)a.refs[at], src.p, src.c)) : 0.0;
        };
        double here;
        auto whole = [&] {
            double all = here = part(lane);
            for (int k = 64 + lane; k < a.nch; k += 64) all += part(k);
            return wave_sum_d(all);
        };
        const double u = uniform_of(a.uniforms[(size_t)n * (a.S + 1) + a.S]);
        double aim = whole();
        if (src.mode != MODE_ROW && aim < LEFT_LEAST) {
            src.whole_row();
            aim = whole();
        }
        aim *= u;
        double before = 0.0, start = 0.0;
        int piece = -1;
        for (int k0 = 0; k0 < a.nch; k0 += 64) {
            const double own = k0 ? part(k0 + lane) : here;
            double s = own;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const double y = __shfl_up(s, o, 64);
                if (lane >= o) s += y;
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
            how = src.mode;
            where = piece;
            rest = aim - start; // to be passed within the piece
            first = 2147483647;
            last = -1;
        }
    }
    __syncthreads();
    const int piece = where;
    if (how == MODE_ROW) src.whole_row();
    if (piece < 0) { // (not where p has a distribution)
        if (tid == 0) emit(-1, 0.f);
        return;
    }
    // places in order, PER of them to a thread
    float z[NG][G];
    double r[NG][G], mine = 0.0;
    const int v0 = piece * VPIECE + tid * PER;
    const bool tail = (piece + 1) * VPIECE > a.V;
    {
        Group<BF> gp[NG], gq[NG];
#pragma unroll
        for (int k = 0; k < NG; ++k) gp[k].load(src.zp, a.V, v0 + k * G);
        if (src.mode == MODE_DIFF) {
#pragma unroll
            for (int k = 0; k < NG; ++k) gq[k].load(src.zq, a.V, v0 + k * G);
        }
#pragma unroll
        for (int k = 0; k < NG; ++k) {
            const int at = Group<BF>::place(a.V, v0 + k * G);
            float w[G] = {};
            gp[k].get(a.V, v0 + k * G, tail, z[k]);
            if (src.mode == MODE_DIFF) gq[k].get(a.V, v0 + k * G, tail, w);
#pragma unroll
            for (int e = 0; e < G; ++e) {
                r[k][e] = at + e == src.x ? 0.0 : src.weight(z[k][e], w[e]);
                mine += r[k][e];
            }
        }
    }
    double upto = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const double y = __shfl_up(upto, o, 64);
        if (lane >= o) upto += y;
    }
    if (lane == 63) ws[tid >> 6] = upto;
    __syncthreads();
    for (int w = 0; w < tid >> 6; ++w) upto += ws[w];
    // the first thread whose end passes `rest` (should rounding leave none, the last with anything), and its place
    if (mine > 0.0) {
        if (upto > rest) atomicMin(&first, tid);
        atomicMax(&last, tid);
    }
    __syncthreads();
    const int who = first != 2147483647 ? first : last;
    if (who < 0 && tid == 0) emit(-1, 0.f); // (as above)
    if (tid != who) return;
    double s = upto - mine;
    int v = -1;
    float at_v = 0.f;
    bool done = false;
#pragma unroll
    for (int k = 0; k < NG; ++k)
#pragma unroll
        for (int e = 0; e < G; ++e) {
            s += r[k][e];
            if (r[k][e] > 0.0 && !done) {
                v = Group<BF>::place(a.V, v0 + k * G) + e;
                at_v = z[k][e];
                done = s > rest;
            }
        }
    emit(v, at_v);
}

hipError_t launch_verify_sums(const VerifyArgs &a, bool bf16, hipStream_t st) {
    const long long rows = (long long)a.N * (a.S + 1) + (a.dlogits ? (long long)a.N * a.S : 0);
    const dim3 grid((unsigned)rows, (unsigned)((a.nch + VT / 64 - 1) / (VT / 64)));
    if (bf16) hipLaunchKernelGGL(verify_sums_kernel<true>, grid, dim3(VT), 0, st, a);
    else hipLaunchKernelGGL(verify_sums_kernel<false>, grid, dim3(VT), 0, st, a);
    return hipGetLastError();
}
hipError_t launch_verify_decide(const VerifyArgs &a, bool bf16, hipStream_t st) {
    if (bf16) hipLaunchKernelGGL(verify_decide_kernel<true>, dim3(a.N), dim3(VT), 0, st, a);
    else hipLaunchKernelGGL(verify_decide_kernel<false>, dim3(a.N), dim3(VT), 0, st, a);
    return hipGetLastError();
}
hipError_t launch_verify_left(const VerifyArgs &a, bool bf16, hipStream_t st) {
    const dim3 grid((unsigned)a.N, (unsigned)a.nch);
    if (bf16) hipLaunchKernelGGL(verify_left_kernel<true>, grid, dim3(VT), 0, st, a);
    else hipLaunchKernelGGL(verify_left_kernel<false>, grid, dim3(VT), 0, st, a);
    return hipGetLastError();
}
hipError_t launch_verify_draw(const VerifyArgs &a, bool bf16, hipStream_t st) {
    if (bf16) hipLaunchKernelGGL(verify_draw_kernel<true>, dim3(a.N), dim3(DT), 0, st, a);
    else hipLaunchKernelGGL(verify_draw_kernel<false>, dim3(a.N), dim3(DT), 0, st, a);
    return hipGetLastError();
}

} // namespace gdn
