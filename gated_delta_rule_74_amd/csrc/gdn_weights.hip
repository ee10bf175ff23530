// Attention weight of every cached row: for the row at position j of sequence n
//
//   w_j = sum over tokens s that see it, heads h, of exp(scale q_sh . row_j - lse_sh)
//
// added to what its slot has gathered so far. The rows are read once where the
// queries of a sequence fit the LDS (twice as many queries: twice); a wave
// takes sixteen rows at a time straight from memory into the operand registers
// of the product, with the next sixteen requested before these are used, and
// the queries as the other operand from LDS. The product is formed as Q K^T: a
// lane then owns one row, adds up the weights of its four queries of a tile,
// and the four lane groups are summed at the end. A lane that has a row alone
// writes its weight: no atomics, and the same order every time.
#include "gdn_serve.hpp"

namespace gdn {

constexpr int WT = 256;           // threads: four waves
constexpr int WROWS = 512;        // rows of a workgroup
constexpr int WLDS = 64 * 1024;   // LDS for queries: two workgroups fit a CU

// 32-column steps the kernel is built for: every number up to six, then even ones
static int weights_ks(int d) {
    const int k = (d + 31) / 32;
    return k <= 6 ? k : (k + 1) / 2 * 2;
}
template <bool BF> __host__ __device__ constexpr int weights_ld(int ks) { return 32 * ks + MLA_PAD<BF>; }
// bytes of a query in LDS, with its statistics
template <bool BF> constexpr int weights_bytes(int ks) { return weights_ld<BF>(ks) * (int)sizeof(typename Op<BF>::S) + 8; }

// KS: 32-column steps of a row; cap: queries held in LDS at once, a multiple of 16
template <bool BF, int KS> __global__ __launch_bounds__(WT, !BF && KS > 12 ? 1 : 2) void mla_weights_kernel(MlaWeightsArgs a, int cap) {
    using S = typename Op<BF>::S;
    extern __shared__ __align__(16) unsigned char weights_lds[];
    S *Q = (S *)weights_lds;
    float *lse2 = (float *)(weights_lds + (size_t)cap * weights_ld<BF>(KS) * sizeof(S)); // in powers of two; +inf: adds nothing
    int *seen = (int *)lse2 + cap;                                       // position of the last row a query sees
    constexpr int V = Op<BF>::VEC, NV = 32 * KS / V, ld = weights_ld<BF>(KS);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15,
              g = lane >> 4;
    const int parts = (int)(((long long)a.cols * a.page + WROWS - 1) / WROWS);
    const int n = blockIdx.x / parts, first = blockIdx.x % parts * WROWS;
    const int len = (int)min((long long)max(a.lens[n], 0), (long long)a.cols * a.page);
    if (first >= len) return;
    const int known = a.known ? a.known[n] : len - a.S;
    const int rows = a.S * a.H, d = a.d;
    const float c2 = a.scale * (float)LOG2E;
    const int *tb = a.table + (size_t)n * a.cols;
    const S *qp = (const S *)a.q + (size_t)n * rows * d;
    // a wave's rows: sixteen at a time, four waves in turn
    const int steps = min(WROWS, len - first + 63) / 64; // (the last may hold rows past the end)
    auto slot_of = [&](int step) { // the row's place in the pool, -1: none
        const int pos = first + step * 64 + wave * 16 + r;
        const int entry = tb[(unsigned)min(pos, len - 1) / (unsigned)a.page];
        return pos < len && (unsigned)entry < (unsigned)a.pages ? entry * a.page + (int)((unsigned)pos % (unsigned)a.page)
                                                                : -1;
    };
    for (int q0 = 0; q0 < rows; q0 += cap) {
        const int nq = min(cap, rows - q0);
        if (q0) lds_barrier(); // the previous queries' readers are done
        for (int e = tid; e < cap * NV; e += WT) {
            const int i = e / NV, c = e % NV * V;
            *reinterpret_cast<u32x4 *>(Q + i * ld + c) =
                load16(i < nq && c < d ? (const void *)(qp + (size_t)(q0 + i) * d + c) : (const void *)&mla_zeros);
        }
        for (int i = tid; i < cap; i += WT) {
            const float l = i < nq ? a.lse[(size_t)n * rows + q0 + i] : -INFINITY;
            lse2[i] = l == -INFINITY ? INFINITY : l * (float)LOG2E;
            seen[i] = i < nq ? len - a.S + (q0 + i) / a.H : -1;
        }
        lds_barrier();
        Frag<BF> K[KS];
        auto fetch = [&](int slot) {
            const S *p = (const S *)a.cache + (size_t)(unsigned)slot * (unsigned)d + 8 * g;
#pragma unroll
            for (int k = 0; k < KS; ++k) K[k] = row8_if(slot >= 0 && 32 * k + 8 * g < d, p + 32 * k);
        };
        int slot = slot_of(0);
        fetch(slot);
        int next = steps > 1 ? slot_of(1) : -1;
        for (int t = 0; t < steps; ++t) {
            const int pos = first + t * 64 + wave * 16 + r, here = slot;
            float old = 0.f;
            if (here >= 0 && g == 0 && (q0 || pos < known)) old = a.weights[here];
            Frag<BF> X[KS];
#pragma unroll
            for (int k = 0; k < KS; ++k) X[k] = K[k];
            slot = next;
            if (t + 1 < steps) {
                fetch(slot);
                next = t + 2 < steps ? slot_of(t + 2) : -1;
            }
            float w = 0.f;
            for (int i = 0; i < nq; i += 16) {
                f32x4 z = zero4();
                const S *qr = Q + (i + r) * ld + 8 * g;
#pragma unroll
                for (int k = 0; k < KS; ++k) z = mma8(row8(qr + 32 * k), X[k], z);
                const f32x4 l2 = *reinterpret_cast<const f32x4 *>(lse2 + i + 4 * g);
                int last[4];
                *reinterpret_cast<u32x4 *>(last) = *reinterpret_cast<const u32x4 *>(seen + i + 4 * g);
#pragma unroll
                for (int e = 0; e < 4; ++e) w += pos <= last[e] ? exp2_fast(fmaf(z[e], c2, -l2[e])) : 0.f;
            }
            w = sum4g(w);
            if (here >= 0 && g == 0) a.weights[here] = (q0 ? old : pos < known ? old * a.decay : 0.f) + w;
        }
    }
}

long long mla_weights_groups(const MlaWeightsArgs &a) {
    return a.N * (((long long)a.cols * a.page + WROWS - 1) / WROWS);
}
template <bool BF, int KS> static hipError_t weights_run(const MlaWeightsArgs &a, hipStream_t st) {
    const long long all = ((long long)a.S * a.H + 15) / 16 * 16, most = WLDS / weights_bytes<BF>(KS) / 16 * 16;
    const int cap = (int)(all < most ? all : most);
    hipLaunchKernelGGL((mla_weights_kernel<BF, KS>), dim3((unsigned)mla_weights_groups(a)), dim3(WT),
                       (unsigned)(cap * weights_bytes<BF>(KS)), st, a, cap);
    return hipGetLastError();
}
template <bool BF> static hipError_t weights_launch(const MlaWeightsArgs &a, hipStream_t st) {
    switch (weights_ks(a.d)) {
    case 1: return weights_run<BF, 1>(a, st);
    case 2: return weights_run<BF, 2>(a, st);
    case 3: return weights_run<BF, 3>(a, st);
    case 4: return weights_run<BF, 4>(a, st);
    case 5: return weights_run<BF, 5>(a, st);
    case 6: return weights_run<BF, 6>(a, st);
    case 8: return weights_run<BF, 8>(a, st);
    case 10: return weights_run<BF, 10>(a, st);
    case 12: return weights_run<BF, 12>(a, st);
    case 14: return weights_run<BF, 14>(a, st);
    case 16: return weights_run<BF, 16>(a, st);
    default: return weights_run<BF, 18>(a, st);
    }
}
hipError_t launch_mla_weights(const MlaWeightsArgs &a, bool bf16, hipStream_t st) {
    return bf16 ? weights_launch<true>(a, st) : weights_launch<false>(a, st);
}

} // namespace gdn
