// New tokens against a paged latent cache (absorbed latent attention).
//
//   z_j = scale q . row_j,  o = sum_j softmax(z)_j row_j[:dl],  lse = log sum_j exp z_j
//
// over the cached rows j of the token's sequence up to its own position. Every
// head of a sequence reads the same rows, so the S * H queries of a sequence
// are the columns of one product and each row is fetched from HBM once per
// 16 * MT of them: a call is bound by the cache's bytes until S * H passes a
// few hundred.
//
// A workgroup takes one sequence, MT * 16 of its queries and one part of its
// length; the parts are joined by mla_join_kernel. Rows go through registers
// (requested one tile ahead, the table entries two) into an LDS tile of
// 32 * WK rows; the four waves split it into WK groups of 32 keys times
// 4 / WK groups of latent columns, each wave with a running softmax of its own
// over its keys, so a tile costs two barriers and no exchange. As in the
// forward pass over expanded heads the products are formed transposed: a lane
// owns one query, and the probabilities are at once the operand of the second
// product, whose other operand is read from the same tile by transposing reads.
#include "gdn_mla.hpp"

namespace gdn {

constexpr float STEP_RAISE = 8.f; // lazy maximum, as in the forward over expanded heads

// Keys [k0, k1) of part `sp` of a sequence of n keys cut into at most nsplit
// parts of whole tiles. The cut follows the sequence's own length, so a short
// sequence in a long table is still spread over several workgroups.
__device__ __forceinline__ int part_keys(int n, int nsplit, int tile) {
    const int per = (n + nsplit - 1) / nsplit;
    return max((per + tile - 1) / tile, 2) * tile;
}

template <bool BF, int DLP, int WK> struct StepShape {
    using S = typename Op<BF>::S;
    static constexpr int DP = DLP + 64, LD = DP + Op<BF>::PAD, KT = 32 * WK, WR = 4 / WK, MV = DLP / 16 / WR,
                         KS = DP / 32, NT = 256, V = Op<BF>::VEC, NIT = KT * (DP / V) / NT;
};

template <bool BF, int DLP, int WK, int MT>
__global__ __launch_bounds__(256, (DLP <= 256 && MT == 1 ? 2 : 1)) void mla_step_kernel(MlaStepArgs a) {
    using P = StepShape<BF, DLP, WK>;
    using S = typename P::S;
    constexpr int TILE_B = P::KT * P::LD * (int)sizeof(S), MERGE_B = 4 * MT * P::MV * P::WR * 64 * 4;
    __shared__ __align__(16) unsigned char smem[TILE_B > MERGE_B ? TILE_B : MERGE_B];
    __shared__ __align__(16) float bias[P::KT];
    __shared__ float Ms[WK][MT * 16], Ss[WK][MT * 16];
    S *T = (S *)smem;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15, g = lane >> 4;
    const int kw = wave % WK, wr = wave / WK;
    const int rows = a.S * a.H, rb = (rows + MT * 16 - 1) / (MT * 16);
    // eight units (sequence, part) side by side on the eight XCDs, then the
    // same units' next block of queries: it finds the rows in its XCD's L2
    const int blk = blockIdx.x / (8 * rb), in = blockIdx.x % (8 * rb);
    const int unit = blk * 8 + in % 8, row0 = (in / 8) * MT * 16;
    if (unit >= a.N * a.nsplit) return;
    const int sp = unit / a.N, nq = unit % a.N;
    const int d = a.dl + a.dr, ng = d / P::V;
    const long long cap = (long long)a.cols * a.page;
    const int n = (int)min((long long)max(a.lens[nq], 0), cap);
    const int per = part_keys(n, a.nsplit, P::KT);
    const int k0 = min((long long)sp * per, (long long)n), k1 = min(k0 + per, n);
    if (k0 >= k1 && a.nsplit > 1) return; // (alone, an empty sequence still writes its zeros)

    // table entries of a tile's rows: lane l holds rows l and (of 128) 64 + l
    const int *tb = a.table + (size_t)nq * a.cols;
    constexpr int NSL = P::KT / 64 > 0 ? P::KT / 64 : 1;
    int pg[NSL];
    auto ask = [&](int t0) {
#pragma unroll
        for (int i = 0; i < NSL; ++i) pg[i] = tb[min(t0 + 64 * i + lane, k1 - 1) / a.page];
    };
    int slot[NSL]; // row of the cache, -1: none (past the part, or an entry outside the pool)
    auto place = [&](int t0) {
#pragma unroll
        for (int i = 0; i < NSL; ++i) {
            const int pos = t0 + 64 * i + lane;
            slot[i] = pos < k1 && (unsigned)pg[i] < (unsigned)a.pages ? pg[i] : -1;
        }
    };
    uint4 reg[P::NIT];
    unsigned long long ok = 0; // bit m: item m lies in a row the part holds
    auto fetch = [&](int t0) {
        ok = 0;
#pragma unroll
        for (int m = 0; m < P::NIT; ++m) {
            const int it = tid + m * P::NT, j = it / ng, c = (it % ng) * P::V;
            int p = __shfl(slot[0], j & 63, 64);
            if (NSL > 1) p = j < 64 ? p : __shfl(slot[NSL - 1], j & 63, 64);
            const bool in_tile = j < P::KT && p >= 0;
            const size_t row = in_tile ? (size_t)p * a.page + (unsigned)(t0 + j) % (unsigned)a.page : 0;
            reg[m] = *reinterpret_cast<const uint4 *>((const S *)a.cache + row * d + c);
            ok |= (in_tile ? 1ull : 0ull) << m;
        }
    };
    const bool any = k0 < k1;
    if (any) {
        ask(k0);
        place(k0);
        fetch(k0);
        ask(k0 + P::KT);
    }
    // queries as operand columns
    Frag<BF> Q[MT][P::KS];
    int see[MT]; // keys below this are seen
    const S *qp = (const S *)a.q + (size_t)nq * rows * d;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int i = row0 + 16 * t + r;
        see[t] = i < rows ? n - a.S + 1 + i / a.H : 0;
#pragma unroll
        for (int k = 0; k < P::KS; ++k) {
            const int c = 32 * k + 8 * g;
            Q[t][k] = (i < rows && c < d) ? row8(qp + (size_t)i * d + c) : zero8<BF>();
        }
    }
    f32x4 O[MT][P::MV];
    float m[MT], l[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        m[t] = -INFINITY;
        l[t] = 0.f;
#pragma unroll
        for (int v = 0; v < P::MV; ++v) O[t][v] = zero4();
    }
    // columns past d are never stored below: zero once
    for (int e = tid; e < P::KT * (P::LD - d); e += P::NT) T[(e / (P::LD - d)) * P::LD + d + e % (P::LD - d)] = S(0);
    const float c2 = a.scale * (float)LOG2E;
    const int all_see = n - a.S + 1; // keys below this are seen by every query
    wait_vmem(); // (q is there: else its first use in the loop waits for the tile in flight)
    for (int t0 = k0; t0 < k1; t0 += P::KT) {
        lds_barrier();
#pragma unroll
        for (int mm = 0; mm < P::NIT; ++mm) {
            const int it = tid + mm * P::NT, j = it / ng, c = (it % ng) * P::V;
            if (j < P::KT)
                *reinterpret_cast<uint4 *>(T + j * P::LD + c) = (ok >> mm) & 1ull ? reg[mm] : uint4{0u, 0u, 0u, 0u};
        }
        if (wave == 0) {
#pragma unroll
            for (int i = 0; i < NSL; ++i)
                if (64 * i + lane < P::KT) bias[64 * i + lane] = slot[i] >= 0 ? 0.f : -INFINITY;
        }
        if (t0 + P::KT < k1) {
            place(t0 + P::KT);
            fetch(t0 + P::KT);
            ask(t0 + 2 * P::KT);
        }
        lds_barrier();
        f32x4 X[MT][2];
#pragma unroll
        for (int t = 0; t < MT; ++t) X[t][0] = X[t][1] = zero4();
#pragma unroll
        for (int k = 0; k < P::KS; ++k) {
            if (32 * k < d) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const Frag<BF> kf = row8(T + (32 * kw + 16 * j + r) * P::LD + 32 * k + 8 * g);
#pragma unroll
                    for (int t = 0; t < MT; ++t) X[t][j] = mma8(kf, Q[t][k], X[t][j]);
                }
            }
        }
        bool raise = false;
        float mx[MT];
        const f32x4 b0 = *reinterpret_cast<const f32x4 *>(bias + 32 * kw + 4 * g);
        const f32x4 b1 = *reinterpret_cast<const f32x4 *>(bias + 32 * kw + 16 + 4 * g);
#pragma unroll
        for (int t = 0; t < MT; ++t) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                X[t][0][e] = b0[e] == 0.f ? X[t][0][e] * c2 : -INFINITY;
                X[t][1][e] = b1[e] == 0.f ? X[t][1][e] * c2 : -INFINITY;
            }
            if (t0 + P::KT > all_see) {
                const int lim = see[t] - t0 - 32 * kw - 4 * g;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    X[t][0][e] = e < lim ? X[t][0][e] : -INFINITY;
                    X[t][1][e] = 16 + e < lim ? X[t][1][e] : -INFINITY;
                }
            }
            float x = X[t][0][0];
#pragma unroll
            for (int e = 0; e < 4; ++e) x = fmaxf(x, fmaxf(X[t][0][e], X[t][1][e]));
            mx[t] = x;
            raise |= x > m[t] + STEP_RAISE;
        }
        if (__any(raise)) {
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const float mn = fmaxf(m[t], max4g(mx[t]));
                const float f = mn == -INFINITY ? 1.f : exp2_fast(m[t] - mn);
                m[t] = mn;
                l[t] *= f;
#pragma unroll
                for (int v = 0; v < P::MV; ++v) O[t][v] *= f;
            }
        }
        Frag<BF> pf[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const float mt = m[t] == -INFINITY ? 0.f : m[t];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                X[t][0][e] = exp2_fast(X[t][0][e] - mt);
                X[t][1][e] = exp2_fast(X[t][1][e] - mt);
            }
            const f32x4 sum = X[t][0] + X[t][1];
            l[t] += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            pf[t] = acc8<BF>(X[t][0], X[t][1]);
        }
#pragma unroll
        for (int v = 0; v < P::MV; ++v) {
            const int c = 16 * (wr * P::MV + v);
            if (c < a.dl) {
                const Frag<BF> vf = col8(T, P::LD, 32 * kw, c, lane);
#pragma unroll
                for (int t = 0; t < MT; ++t) O[t][v] = mma8(vf, pf[t], O[t][v]);
            }
        }
    }
    // join the key groups: common maximum, then the rescaled sums one group after the other
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        l[t] = sum4g(l[t]);
        if (wr == 0 && g == 0) {
            Ms[kw][16 * t + r] = m[t];
            Ss[kw][16 * t + r] = l[t];
        }
    }
    lds_barrier();
    float ml[MT], sl[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        float mm = Ms[0][16 * t + r];
#pragma unroll
        for (int w = 1; w < WK; ++w) mm = fmaxf(mm, Ms[w][16 * t + r]);
        float sm = 0.f;
#pragma unroll
        for (int w = 0; w < WK; ++w) {
            const float mw = Ms[w][16 * t + r];
            sm += mw == -INFINITY ? 0.f : Ss[w][16 * t + r] * exp2_fast(mw - mm);
        }
        const float f = m[t] == -INFINITY ? 0.f : exp2_fast(m[t] - mm);
#pragma unroll
        for (int v = 0; v < P::MV; ++v) O[t][v] *= f;
        ml[t] = mm;
        sl[t] = sm;
    }
    f32x4 *X = (f32x4 *)smem + wr * MT * P::MV * 64;
#pragma unroll
    for (int w = 1; w < WK; ++w) {
        if (kw == w) {
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int v = 0; v < P::MV; ++v) X[(t * P::MV + v) * 64 + lane] = O[t][v];
        }
        lds_barrier();
        if (kw == 0) {
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int v = 0; v < P::MV; ++v) O[t][v] += X[(t * P::MV + v) * 64 + lane];
        }
        if (w + 1 < WK) lds_barrier();
    }
    if (kw != 0) return;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int i = row0 + 16 * t + r;
        if (i >= rows) continue;
        const size_t row = (size_t)nq * rows + i;
        const float inv = sl[t] != 0.f ? 1.f / sl[t] : 0.f;
#pragma unroll
        for (int v = 0; v < P::MV; ++v) {
            const int c = 16 * (wr * P::MV + v) + 4 * g;
            if (c >= a.dl) continue;
            if (a.nsplit > 1) store4(a.part + (row * a.nsplit + sp) * a.dl + c, O[t][v]);
            else store4((S *)a.o + row * a.dl + c, O[t][v] * inv);
        }
        if (wr == 0 && g == 0) {
            if (a.nsplit > 1) {
                a.part_ml[(row * a.nsplit + sp) * 2] = ml[t];
                a.part_ml[(row * a.nsplit + sp) * 2 + 1] = sl[t];
            } else if (a.lse) {
                a.lse[row] = sl[t] == 0.f ? -INFINITY : (ml[t] + __builtin_amdgcn_logf(sl[t])) * 0.69314718055994531f;
            }
        }
    }
}

// Joins the parts of a sequence: o = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i,
// in part order within each of 16 interleaved groups, then over the groups. A
// workgroup takes one query and 64 columns.
template <bool BF> __global__ __launch_bounds__(256) void mla_join_kernel(MlaStepArgs a, int tile) {
    using S = typename Op<BF>::S;
    __shared__ float red[4], wgt[MLA_SPLIT_MAX];
    __shared__ __align__(16) f32x4 acc[16][16];
    const int tid = threadIdx.x, rows = a.S * a.H, lane = tid & 63, wave = tid >> 6;
    const size_t row = blockIdx.x;
    const int nq = blockIdx.x / rows;
    const int n = (int)min((long long)max(a.lens[nq], 0), (long long)a.cols * a.page);
    const int per = part_keys(n, a.nsplit, tile), cnt = (n + per - 1) / per;
    const float *ml = a.part_ml + row * a.nsplit * 2;
    float m = -INFINITY;
    for (int i = tid; i < cnt; i += 256) m = fmaxf(m, ml[2 * i]);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
    if (lane == 0) red[wave] = m;
    __syncthreads();
    m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    __syncthreads();
    float l = 0.f;
    for (int i = tid; i < cnt; i += 256) {
        const float w = ml[2 * i] == -INFINITY ? 0.f : exp2_fast(ml[2 * i] - m);
        wgt[i] = w;
        l += w * ml[2 * i + 1];
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) l += __shfl_xor(l, o, 64);
    if (lane == 0) red[wave] = l;
    __syncthreads();
    l = (red[0] + red[1]) + (red[2] + red[3]);
    const int c = blockIdx.y * 64 + (tid & 15) * 4, grp = tid >> 4;
    f32x4 x = zero4();
    if (c < a.dl) {
        const float *p = a.part + row * a.nsplit * a.dl + c;
        for (int i = grp; i < cnt; i += 16)
            if (wgt[i] != 0.f) x += *reinterpret_cast<const f32x4 *>(p + (size_t)i * a.dl) * wgt[i];
    }
    acc[grp][tid & 15] = x;
    __syncthreads();
    if (grp == 0 && c < a.dl) {
        for (int i = 1; i < 16; ++i) x += acc[i][tid & 15];
        store4((S *)a.o + row * a.dl + c, x * (l != 0.f ? 1.f / l : 0.f));
    }
    if (a.lse && blockIdx.y == 0 && tid == 0)
        a.lse[row] = l == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f;
}

static int step_class(int dl) { return dl <= 64 ? 64 : dl <= 128 ? 128 : dl <= 256 ? 256 : 512; }
// key groups: 32 * WK rows per tile, so that a tile in flight fits the registers
static int step_wk(int dl, bool bf16) { return bf16 ? (dl <= 128 ? 4 : 2) : dl <= 64 ? 4 : dl <= 256 ? 2 : 1; }

void mla_step_plan(MlaStepArgs &a, bool bf16, int cus) {
    const long long rows = (long long)a.S * a.H;
    // query blocks per workgroup: two where the registers hold them (fp32
    // operands and the widest latent take twice the registers)
    a.mt = rows > 16 && bf16 && a.dl <= 256 ? 2 : 1;
    const long long rb = (rows + 16 * a.mt - 1) / (16 * a.mt), tile = 32 * step_wk(a.dl, bf16);
    const long long cap = (long long)a.cols * a.page, want = (4LL * cus + a.N * rb - 1) / (a.N * rb);
    long long n = (cap + 2 * tile - 1) / (2 * tile);
    if (n > want) n = want;
    if (n > MLA_SPLIT_MAX) n = MLA_SPLIT_MAX;
    a.nsplit = n < 1 ? 1 : (int)n;
}

template <bool BF, int DLP, int WK, int MT> static hipError_t step_run(const MlaStepArgs &a, hipStream_t st) {
    const long long rb = ((long long)a.S * a.H + MT * 16 - 1) / (MT * 16), units = ((long long)a.N * a.nsplit + 7) / 8 * 8;
    hipLaunchKernelGGL((mla_step_kernel<BF, DLP, WK, MT>), dim3((unsigned)(units * rb)), dim3(256), 0, st, a);
    return hipGetLastError();
}
template <bool BF, int DLP, int WK> static hipError_t step_rows(const MlaStepArgs &a, hipStream_t st) {
    if constexpr (BF && DLP <= 256)
        if (a.mt == 2) return step_run<BF, DLP, WK, 2>(a, st);
    return step_run<BF, DLP, WK, 1>(a, st);
}
template <bool BF> static hipError_t step_launch(const MlaStepArgs &a, hipStream_t st) {
    switch (step_class(a.dl)) {
    case 64: return step_rows<BF, 64, 4>(a, st);
    case 128: return step_rows<BF, 128, BF ? 4 : 2>(a, st);
    case 256: return step_rows<BF, 256, 2>(a, st);
    default: return step_rows<BF, 512, BF ? 2 : 1>(a, st);
    }
}
hipError_t launch_mla_step(const MlaStepArgs &a, bool bf16, hipStream_t st) {
    return bf16 ? step_launch<true>(a, st) : step_launch<false>(a, st);
}

hipError_t launch_mla_join(const MlaStepArgs &a, bool bf16, hipStream_t st) {
    const dim3 grid((unsigned)((long long)a.N * a.S * a.H), (unsigned)((a.dl + 63) / 64));
    const int tile = 32 * step_wk(a.dl, bf16);
    if (bf16) hipLaunchKernelGGL(mla_join_kernel<true>, grid, dim3(256), 0, st, a, tile);
    else hipLaunchKernelGGL(mla_join_kernel<false>, grid, dim3(256), 0, st, a, tile);
    return hipGetLastError();
}

} // namespace gdn
