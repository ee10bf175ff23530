// Attention weight of every cached row: for the row at position j of sequence n
//
//   w_j = sum over tokens s that see it, heads h, of exp(scale q_sh . row_j - lse_sh)
//
// added to what its slot has gathered so far. The rows are read once, straight
// from memory into the operand registers of the product; the queries are the
// other operand, from LDS. The product is formed as Q K^T: a lane then owns one
// row, adds up the weights of its four queries of a tile, and the four lane
// groups are summed at the end. A lane that has a row alone writes its weight:
// no atomics, and the same order every time.
// Few queries (they fit 64 KB of LDS): all of them stay there while a wave walks
// its rows, sixteen at a time, the next sixteen requested before these are
// used; bound by the cache's bytes (256 sequences of up to 4096 rows of 160 bf16, 16
// queries: 37 us, 4.7 TB/s; a call takes 50 us, and 61 with runs that are not laid end to end
// over the chip). More: a wave keeps 16 (bf16: 32) rows and the queries pass by, 32 at a
// time, in two buffers; bound by the products (12 prompts of up to 2000 rows of 320
// fp32, 256 queries: 31 us; the way of few queries: 300).
#include "gdn_lds_tile.hpp"
#include "gdn_serve.hpp"

namespace gdn {

constexpr int WT = 256;           // threads: four waves
constexpr int WLDS = 64 * 1024;   // LDS for queries: two workgroups fit a CU

// 32-column steps the kernel is built for: every number up to six, then even ones
static int weights_ks(int d) {
    const int k = (d + 31) / 32;
    return k <= 6 ? k : (k + 1) / 2 * 2;
}
template <bool BF> __host__ __device__ constexpr int weights_ld(int ks) { return 32 * ks + MLA_PAD<BF>; }
// bytes of a query in LDS, with its statistics
template <bool BF> constexpr int weights_bytes(int ks) { return weights_ld<BF>(ks) * (int)sizeof(typename Op<BF>::S) + 8; }

// Rows of a workgroup: a quarter of them is a wave's run, whose table entries are read together.
// Long runs pay for a workgroup's start, short ones fill the chip where there are few rows.
static int weights_rows(const MlaWeightsArgs &a) {
    const long long cap = (long long)a.cols * a.page;
    int rows = 512;
    while (rows > 64 && a.N * ((cap + rows - 1) / rows) < 1024) rows /= 2;
    return rows;
}

__device__ __forceinline__ int weights_len(const MlaWeightsArgs &a, int n) {
    return (int)min((long long)max(a.lens[n], 0), (long long)a.cols * a.page);
}
__device__ __forceinline__ int weights_parts(const MlaWeightsArgs &a, int n, int rows) {
    return (weights_len(a, n) + rows - 1) / rows;
}

// KS: 32-column steps of a row; cap: the queries, rounded up to a multiple of
// 16; run: rows of a wave, a multiple of 16 up to 128
template <bool BF, int KS>
__global__ __launch_bounds__(WT, !BF && KS > 12 ? 1 : 2) void mla_weights_kernel(MlaWeightsArgs a, int cap, int run) {
    using S = typename Op<BF>::S;
    extern __shared__ __align__(16) unsigned char weights_lds[];
    S *Q = (S *)weights_lds;
    float *lse2 = (float *)(weights_lds + (size_t)cap * weights_ld<BF>(KS) * sizeof(S)); // in powers of two; +inf: adds nothing
    int *seen = (int *)lse2 + cap;                                       // position of the last row a query sees
    constexpr int V = Op<BF>::VEC, NV = 32 * KS / V, ld = weights_ld<BF>(KS);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15,
              g = lane >> 4;
    int n, first;
    if (!find_piece(a.N, [&](int i) { return weights_parts(a, i, 4 * run); }, blockIdx.x, lane, n, first)) return;
    first *= 4 * run;
    const int len = weights_len(a, n);
    const int known = a.known ? a.known[n] : len - a.S;
    const int rows = a.S * a.H, d = a.d;
    const float c2 = a.scale * (float)LOG2E;
    const int *tb = a.table + (size_t)n * a.cols;
    const S *qp = (const S *)a.q + (size_t)n * rows * d;
    // the wave's rows: their places in the pool (-1: none), two to a lane
    const int mine = first + wave * run, steps = max(0, min(run, len - mine) + 15) / 16;
    int place[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) place[i] = tb[(unsigned)min(mine + 64 * i + lane, len - 1) / (unsigned)a.page];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int pos = mine + 64 * i + lane;
        place[i] = pos < len && (unsigned)place[i] < (unsigned)a.pages
                       ? place[i] * a.page + (int)((unsigned)pos % (unsigned)a.page)
                       : -1;
    }
    auto slot_of = [&](int t) { return __shfl(t < 4 ? place[0] : place[1], (t & 3) * 16 + r, 64); };
    Frag<BF> K[KS];
    auto fetch = [&](int slot) {
        const S *p = (const S *)a.cache + (size_t)(unsigned)slot * (unsigned)d + 8 * g;
#pragma unroll
        for (int k = 0; k < KS; ++k) K[k] = row8_if(slot >= 0 && 32 * k + 8 * g < d, p + 32 * k);
    };
    int slot = slot_of(0);
    if (steps > 0) fetch(slot);
    constexpr int NB = 8; // pieces of a thread, requested together
    for (int e0 = tid; e0 < cap * NV; e0 += NB * WT) {
        u32x4 x[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int e = e0 + b * WT, i = e / NV, c = e % NV * V;
            x[b] = load16(i < rows && c < d ? (const void *)(qp + (size_t)i * d + c) : (const void *)&mla_zeros);
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const int e = e0 + b * WT;
            if (e < cap * NV) *reinterpret_cast<u32x4 *>(Q + e / NV * ld + e % NV * V) = x[b];
        }
    }
    for (int i = tid; i < cap; i += WT) {
        const float l = i < rows ? a.lse[(size_t)n * rows + i] : -INFINITY;
        lse2[i] = l == -INFINITY ? INFINITY : l * (float)LOG2E;
        seen[i] = i < rows ? len - a.S + i / a.H : -1;
    }
    lds_barrier();
    for (int t = 0; t < steps; ++t) {
        const int pos = mine + t * 16 + r, here = slot;
        const bool keep = here >= 0 && g == 0;
        const float old = keep && pos < known ? a.weights[here] * a.decay : 0.f;
        Frag<BF> X[KS];
#pragma unroll
        for (int k = 0; k < KS; ++k) X[k] = K[k];
        if (t + 1 < steps) {
            slot = slot_of(t + 1);
            fetch(slot);
        }
        float w = 0.f;
        auto add_up = [&](const f32x4 &z, int i) {
            const f32x4 l2 = *reinterpret_cast<const f32x4 *>(lse2 + i + 4 * g);
            int last[4];
            *reinterpret_cast<u32x4 *>(last) = *reinterpret_cast<const u32x4 *>(seen + i + 4 * g);
#pragma unroll
            for (int e = 0; e < 4; ++e) w += pos <= last[e] ? exp2_fast(fmaf(z[e], c2, -l2[e])) : 0.f;
        };
        // two tiles of queries at a time: two sums of products that do not wait for each other
        int i = 0;
        for (; i + 16 < rows; i += 32) {
            f32x4 z = zero4(), y = zero4();
            const S *qr = Q + (i + r) * ld + 8 * g;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                z = mma8(row8(qr + 32 * k), X[k], z);
                y = mma8(row8(qr + 16 * ld + 32 * k), X[k], y);
            }
            add_up(z, i);
            add_up(y, i + 16);
        }
        if (i < rows) {
            f32x4 z = zero4();
            const S *qr = Q + (i + r) * ld + 8 * g;
#pragma unroll
            for (int k = 0; k < KS; ++k) z = mma8(row8(qr + 32 * k), X[k], z);
            add_up(z, i);
        }
        w = sum4g(w);
        if (keep) a.weights[here] = old + w;
    }
}

// Many queries, QS at a time; RT: tiles of 16 rows a wave keeps.
template <bool BF> constexpr int WEIGHTS_RT = BF ? 2 : 1;
constexpr int QS = 32;
template <bool BF, int KS> __global__ __launch_bounds__(WT, !BF && KS > 12 ? 1 : 2) void mla_weights_many_kernel(MlaWeightsArgs a) {
    using S = typename Op<BF>::S;
    using P = LdsTile<BF, KS>;
    constexpr int RT = WEIGHTS_RT<BF>, NL = QS * P::RU / WT, NQ = QS / 16; // loads of a thread; tiles of queries
    __shared__ u32x4 T[2][QS * P::RU];
    __shared__ __align__(16) float lse2[2][QS];
    __shared__ __align__(16) int seen[2][QS];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15,
              g = lane >> 4;
    int n, first;
    if (!find_piece(a.N, [&](int i) { return weights_parts(a, i, 64 * RT); }, blockIdx.x, lane, n, first)) return;
    first *= 64 * RT;
    const int len = weights_len(a, n);
    const int known = a.known ? a.known[n] : len - a.S;
    const int rows = a.S * a.H, d = a.d, stages = (rows + QS - 1) / QS;
    const float c2 = a.scale * (float)LOG2E;
    const int *tb = a.table + (size_t)n * a.cols;
    const S *qp = (const S *)a.q + (size_t)n * rows * d;
    // the query of the QS that a load takes, and its column (past d: from the zeros)
    int place[NL];
#pragma unroll
    for (int j = 0; j < NL; ++j) {
        const int x = (wave * NL + j) * 64 + lane, q = x / P::RU, c = (x % P::RU ^ (q & P::XM)) * P::V;
        place[j] = q << 16 | (c < d ? c : 0xffff);
    }
    auto fetch = [&](int s) { // QS queries into buffer s & 1 (past the last: that one again, not counted below)
#pragma unroll
        for (int j = 0; j < NL; ++j) {
            const int i = min(QS * s + (place[j] >> 16), rows - 1), c = place[j] & 0xffff;
            const S *src = qp + (size_t)(unsigned)i * (unsigned)d + c;
            load_to_lds(c != 0xffff ? (const void *)src : (const void *)&mla_zeros,
                        lds_place(T[s & 1] + (wave * NL + j) * 64));
        }
    };
    auto lse_of = [&](int i) { return i < rows ? a.lse[(size_t)n * rows + i] : -INFINITY; };
    auto put = [&](int s, float l) {
        lse2[s & 1][tid] = l == -INFINITY ? INFINITY : l * (float)LOG2E;
        seen[s & 1][tid] = QS * s + tid < rows ? len - a.S + (QS * s + tid) / a.H : -1;
    };
    fetch(0);
    // the wave's rows, from memory into operand registers
    int slot[RT];
    Frag<BF> X[RT][KS];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int pos = first + (wave * RT + t) * 16 + r, entry = tb[(unsigned)min(pos, len - 1) / (unsigned)a.page];
        slot[t] = pos < len && (unsigned)entry < (unsigned)a.pages ? entry * a.page + (int)((unsigned)pos % (unsigned)a.page) : -1;
        const S *p = (const S *)a.cache + (size_t)(unsigned)slot[t] * (unsigned)d + 8 * g;
#pragma unroll
        for (int k = 0; k < KS; ++k) X[t][k] = row8_if(slot[t] >= 0 && 32 * k + 8 * g < d, p + 32 * k);
    }
    if (tid < QS) put(0, lse_of(tid));
    TileReads<P> at;
    at.init(lane);
    float w[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) w[t] = 0.f;
    wait_vmem();
    lds_barrier();
    for (int s = 0; s < stages; ++s) {
        float l = 0.f;
        if (s + 1 < stages) {
            fetch(s + 1); // (its buffer's last readers passed the barrier before this stage)
            if (tid < QS) l = lse_of(QS * (s + 1) + tid);
        }
        f32x4 z[NQ][RT];
#pragma unroll
        for (int i = 0; i < NQ; ++i)
#pragma unroll
            for (int t = 0; t < RT; ++t) z[i][t] = zero4();
        // operands a step ahead of the products that take them
        Frag<BF> qf[2][NQ];
        auto ahead = [&](int k) {
#pragma unroll
            for (int i = 0; i < NQ; ++i) qf[k & 1][i] = at.rows(T[s & 1], 16 * i, k);
        };
        ahead(0);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            if (k + 1 < KS) ahead(k + 1);
            in_flight();
#pragma unroll
            for (int i = 0; i < NQ; ++i)
#pragma unroll
                for (int t = 0; t < RT; ++t) z[i][t] = mma8(qf[k & 1][i], X[t][k], z[i][t]);
            in_flight();
        }
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            const f32x4 l2 = *reinterpret_cast<const f32x4 *>(&lse2[s & 1][16 * i + 4 * g]);
            int last[4];
            *reinterpret_cast<u32x4 *>(last) = *reinterpret_cast<const u32x4 *>(&seen[s & 1][16 * i + 4 * g]);
#pragma unroll
            for (int t = 0; t < RT; ++t) {
                const int pos = first + (wave * RT + t) * 16 + r;
#pragma unroll
                for (int e = 0; e < 4; ++e) w[t] += pos <= last[e] ? exp2_fast(fmaf(z[i][t][e], c2, -l2[e])) : 0.f;
            }
        }
        if (s + 1 < stages && tid < QS) put(s + 1, l);
        wait_vmem(); // the next queries are in LDS
        lds_barrier();
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int pos = first + (wave * RT + t) * 16 + r;
        w[t] = sum4g(w[t]);
        if (slot[t] >= 0 && g == 0) a.weights[slot[t]] = (pos < known ? a.weights[slot[t]] * a.decay : 0.f) + w[t];
    }
}

// queries that stay in LDS
template <bool BF> constexpr int weights_cap(int ks) { return WLDS / weights_bytes<BF>(ks) / 16 * 16; }
static bool weights_many(const MlaWeightsArgs &a, bool bf16) {
    const int ks = weights_ks(a.d);
    return (long long)a.S * a.H > (bf16 ? weights_cap<true>(ks) : weights_cap<false>(ks));
}
long long mla_weights_groups(const MlaWeightsArgs &a, bool bf16) {
    const int rows = !weights_many(a, bf16) ? weights_rows(a) : 64 * (bf16 ? WEIGHTS_RT<true> : WEIGHTS_RT<false>);
    return a.N * (((long long)a.cols * a.page + rows - 1) / rows);
}
template <bool BF, int KS> static hipError_t weights_run(const MlaWeightsArgs &a, hipStream_t st) {
    const dim3 grid((unsigned)mla_weights_groups(a, BF));
    if (weights_many(a, BF)) {
        hipLaunchKernelGGL((mla_weights_many_kernel<BF, KS>), grid, dim3(WT), 0, st, a);
        return hipGetLastError();
    }
    const int cap = (a.S * a.H + 15) / 16 * 16;
    hipLaunchKernelGGL((mla_weights_kernel<BF, KS>), grid, dim3(WT), (unsigned)(cap * weights_bytes<BF>(KS)), st, a, cap,
                       weights_rows(a) / 4);
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
