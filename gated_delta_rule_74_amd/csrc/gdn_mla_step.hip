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
// A workgroup takes MT * 16 queries and an equal share of the cached rows; the
// parts of a sequence are joined by mla_join_kernel. Rows go through registers
// (requested one tile ahead, the table entries two) into an LDS tile of 64 rows
// (32 beyond 256 latent columns); the four waves split it into WK groups of KW
// keys (16 or 32, see StepShape) times 4 / WK groups of latent columns, each
// wave with a running softmax of its own over its keys, so a tile costs two
// barriers and no exchange. As in the
// forward pass over expanded heads the products are formed transposed: a lane
// owns one query, and the probabilities are at once the operand of the second
// product, whose other operand is read from the same tile by transposing reads.
// Bound by the cache's bytes with what a workgroup has in flight (two or three
// waves per SIMD, a tile each): 256 sequences of 0 to 4096 rows of 128 + 32
// bf16 in 34 us and 6 us for the join, 4.9 TB/s where a large copy reaches 5.6;
// one of 131072 rows of 512 + 64 in 32 us and 12 us, 4.7 TB/s. In fp32 by the
// matrix products (48 drafts of three tokens up to 1500 rows, 8 heads of
// 256 + 64: 38 us).
#include "gdn_mla.hpp"

namespace gdn {

constexpr float STEP_RAISE = 8.f; // lazy maximum, as in the forward over expanded heads

// How the cached rows are shared out. The sequences' tiles (2^MlaStepArgs::tile rows),
// end to end, are cut into equal shares, one per workgroup, whatever the single
// lengths are: a batch of 256 lengths from 0 to 4096 took 51 us with each
// sequence cut into four equal parts (some CUs had twice the work of others).
// A workgroup walks the pieces of one or more sequences; a sequence it holds
// whole it finishes, of others it leaves a part. Only the first and the last
// piece of a share can be parts, which gives each workgroup two places to
// leave them.
// where workgroup w leaves its part of a sequence whose tiles begin at `begin`
__device__ __forceinline__ int part_slot(int w, int begin, int share) { return 2 * w + (begin > w * share ? 1 : 0); }

// A tile holds KT rows; a wave takes KW of them (32 bf16 rows fill one MFMA's
// K, 16 fp32 rows four) and DLP / WR columns. In bf16 two key groups times two
// column groups: the scores are formed twice, which is nothing beside the
// memory, and leaves a wave few enough registers for two or three waves per
// SIMD; those hide a piece's start and end. In fp32 the products are what takes
// the time (a sixteenth of the bf16 rate), so up to 256 columns four key groups
// form each score once (8 sequences of 30000 rows of 256 + 64, 32 queries: 104
// us with two groups, 85 with four); beyond, the accumulators of all columns do
// not fit a wave.
constexpr int step_tile(int dlp) { return dlp <= 256 ? 6 : 5; } // log2 of a tile's rows, by padded columns
template <bool BF, int DLP, int MT> struct StepShape {
    using S = typename Op<BF>::S;
    static constexpr int WK = !BF && DLP <= 256 ? 4 : 2, WR = 4 / WK, KW = BF && DLP <= 256 ? 32 : 16, KT = KW * WK,
                         NJ = KW / 16, NT = 256, V = Op<BF>::VEC, DP = DLP + 64, LD = DP + MLA_PAD<BF>,
                         MV = DLP / 16 / WR, MP = MV / WK, KS = DP / 32, RP = NT / (DP / V) > 0 ? NT / (DP / V) : 1,
                         NIT = (KT + RP - 1) / RP, TILE_B = KT * LD * (int)sizeof(S), MERGE_B = 4 * MT * MP * 64 * 16;
    // The queries' operands stay in registers where those hold them without
    // crowding the rows in flight, else in LDS (bf16 256 + 64, 32 queries, as
    // above: 56 us in registers, 36 in LDS; 512 + 64, 16 queries, 200 sequences
    // up to 1000 rows: 53 and 49).
    static constexpr bool QL = !BF || DLP * MT >= 256;
    static_assert(KT == 1 << step_tile(DLP), "shares are cut between tiles");
};

typedef short short8_t __attribute__((ext_vector_type(8)));

// One more product over the NJ * 16 rows of an accumulator-ordered operand pair.
template <int NJ> __device__ __forceinline__ f32x4 mma_rows(const Frag<true> &a, const Frag<true> &b, f32x4 c) {
    if constexpr (NJ == 2) return mma8(a, b, c);
    const short8_t x = __builtin_bit_cast(short8_t, a.v), y = __builtin_bit_cast(short8_t, b.v);
    return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_shufflevector(x, x, 0, 1, 2, 3),
                                                     __builtin_shufflevector(y, y, 0, 1, 2, 3), c, 0, 0, 0);
}
template <int NJ> __device__ __forceinline__ f32x4 mma_rows(const Frag<false> &a, const Frag<false> &b, f32x4 c) {
    static_assert(NJ == 1, "an fp32 wave takes 16 rows");
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.lo[j], b.lo[j], c, 0, 0, 0);
    return c;
}
template <int NJ> __device__ __forceinline__ Frag<true> col_rows(const u16 *X, int ld, int k0, int m0, int lane) {
    if constexpr (NJ == 2) return col8(X, ld, k0, m0, lane);
    const short4_t x = operand_tr4(X, ld, k0, m0, lane);
    return {join8(x, x)};
}
template <int NJ> __device__ __forceinline__ Frag<false> col_rows(const float *X, int ld, int k0, int m0, int lane) {
    const float *p = X + (k0 + 4 * (lane >> 4)) * ld + m0 + (lane & 15);
    Frag<false> f;
#pragma unroll
    for (int e = 0; e < 4; ++e) f.lo[e] = p[e * ld];
    return f;
}

// Rows [k0, k1e) of sequence nq for the queries from row0 on (k1e may pass its
// end); slot: where to leave the part, -1: all of the sequence, finish it.
template <bool BF, int DLP, int MT>
__device__ __forceinline__ void step_piece(const MlaStepArgs a, int nq, int k0, int k1e, int row0, int slot,
                                           unsigned char *smem, typename Op<BF>::S *Qs, float *bias, float *Ms,
                                           float *Ss) {
    using P = StepShape<BF, DLP, MT>;
    using S = typename P::S;
    S *T = (S *)smem;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15,
              g = lane >> 4;
    const int kw = wave % P::WK, wr = wave / P::WK, rows = a.S * a.H;
    const int d = a.dl + a.dr, ng = d / P::V, rp = P::NT / ng;
    const int n = seq_rows(a, nq), k1 = min(k1e, n);

    // the table entry and the cache row of tile row `lane`, requested two tiles
    // and known one tile ahead; -1: no row (past the part, or an entry outside
    // the pool)
    const int *tb = a.table + (size_t)nq * a.cols;
    int entry = -1, row = -1;
    auto ask = [&](int t0) {
        if (lane < P::KT) entry = tb[(unsigned)min(t0 + lane, k1 - 1) / (unsigned)a.page];
    };
    auto place = [&](int t0) {
        const int pos = t0 + lane;
        row = lane < P::KT && pos < k1 && (unsigned)entry < (unsigned)a.pages
                  ? entry * a.page + (int)((unsigned)pos % (unsigned)a.page)
                  : -1;
    };
    // a thread loads one 16-byte column of every rp-th row of a tile
    const int j0 = tid < rp * ng ? tid / ng : P::KT, c0 = (tid % ng) * P::V;
    u32x4 reg[P::NIT];
    auto fetch = [&] {
#pragma unroll
        for (int m = 0; m < P::NIT; ++m) {
            const int j = j0 + m * rp, p = __shfl(row, j & 63, 64);
            // (no row: zeros, chosen by address, so that nothing waits for the load here)
            const S *src = (const S *)a.cache + (size_t)(unsigned)p * (unsigned)d + c0;
            reg[m] = load16(j < P::KT && p >= 0 ? src : (const S *)&mla_zeros);
        }
    };
    ask(k0);
    place(k0);
    fetch();
    // queries as operand columns
    Frag<BF> Q[P::QL ? 1 : MT][P::KS];
    int see[MT]; // keys below this are seen
    const S *qp = (const S *)a.q + (size_t)nq * rows * d;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int i = row0 + 16 * t + r;
        see[t] = i < rows ? n - a.S + 1 + i / a.H : 0;
        if constexpr (!P::QL) {
#pragma unroll
            for (int k = 0; k < P::KS; ++k) {
                const int c = 32 * k + 8 * g;
                Q[t][k] = row8_if(i < rows && c < d, qp + (size_t)i * d + c);
            }
        }
    }
    if constexpr (P::QL) {
        lds_barrier(); // (the previous piece's readers are done)
        constexpr int NV = P::DP / P::V, NQ = (MT * 16 * NV + P::NT - 1) / P::NT;
        u32x4 x[NQ]; // all requested before the first is waited for
#pragma unroll
        for (int k = 0; k < NQ; ++k) {
            const int e = tid + k * P::NT, i = row0 + e / NV, c = e % NV * P::V;
            x[k] = load16(e < MT * 16 * NV && i < rows && c < d ? (const void *)(qp + (size_t)i * d + c)
                                                                : (const void *)&mla_zeros);
        }
#pragma unroll
        for (int k = 0; k < NQ; ++k) {
            const int e = tid + k * P::NT;
            if (e < MT * 16 * NV) *reinterpret_cast<u32x4 *>(Qs + e / NV * P::LD + e % NV * P::V) = x[k];
        }
    }
    lds_barrier(); // (the previous piece's readers are done)
    // columns past d are never stored below: zero once
    for (int w = (P::DP - d) / P::V, e = tid; e < P::KT * w; e += P::NT)
        *reinterpret_cast<u32x4 *>(T + e / w * P::LD + d + e % w * P::V) = u32x4{0u, 0u, 0u, 0u};
    f32x4 O[MT][P::MV];
    float m[MT], l[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        m[t] = -INFINITY;
        l[t] = 0.f;
#pragma unroll
        for (int v = 0; v < P::MV; ++v) O[t][v] = zero4();
    }
    const float c2 = a.scale * (float)LOG2E;
    wait_vmem(); // (what is held is there: else its first use in the loop waits for the tile in flight)
    ask(k0 + P::KT);
    for (int t0 = k0; t0 < k1; t0 += P::KT) {
        lds_barrier(); // the previous tile's readers (or the zeros' writers) are done
#pragma unroll
        for (int mm = 0; mm < P::NIT; ++mm) {
            const int j = j0 + mm * rp;
            if (j < P::KT) *reinterpret_cast<u32x4 *>(T + j * P::LD + c0) = reg[mm];
        }
        if (wave == 0 && lane < P::KT) bias[lane] = row >= 0 ? 0.f : -INFINITY;
        if (t0 + P::KT < k1) {
            place(t0 + P::KT);
            ask(t0 + 2 * P::KT);
            fetch();
        }
        lds_barrier();
        f32x4 X[MT][P::NJ];
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int j = 0; j < P::NJ; ++j) X[t][j] = zero4();
        const S *kr = T + (P::KW * kw + r) * P::LD + 8 * g;
#pragma unroll
        for (int k = 0; k < P::KS; ++k) {
            Frag<BF> qf[MT];
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                if constexpr (P::QL) qf[t] = row8(Qs + (16 * t + r) * P::LD + 32 * k + 8 * g);
                else qf[t] = Q[t][k];
            }
#pragma unroll
            for (int j = 0; j < P::NJ; ++j) {
                const Frag<BF> kf = row8(kr + 16 * j * P::LD + 32 * k);
#pragma unroll
                for (int t = 0; t < MT; ++t) X[t][j] = mma8(kf, qf[t], X[t][j]);
            }
        }
        bool raise = false;
        float mx[MT];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            mx[t] = -INFINITY;
#pragma unroll
            for (int j = 0; j < P::NJ; ++j) {
                const f32x4 bj = *reinterpret_cast<const f32x4 *>(bias + P::KW * kw + 16 * j + 4 * g);
                // Masked on every tile, without a branch: the compiler (ROCm 7.2) leaves out the wait states
                // between an MFMA and a use of its result behind a conditional block that follows it at once.
                const int lim = see[t] - t0 - P::KW * kw - 16 * j - 4 * g;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    X[t][j][e] = e < lim && bj[e] == 0.f ? X[t][j][e] * c2 : -INFINITY;
#pragma unroll
                for (int e = 0; e < 4; ++e) mx[t] = fmaxf(mx[t], X[t][j][e]);
            }
            raise |= mx[t] > m[t] + STEP_RAISE;
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
            for (int j = 0; j < P::NJ; ++j) {
#pragma unroll
                for (int e = 0; e < 4; ++e) X[t][j][e] = exp2_fast(X[t][j][e] - mt);
                l[t] += (X[t][j][0] + X[t][j][1]) + (X[t][j][2] + X[t][j][3]);
            }
            pf[t] = acc8<BF>(X[t][0], X[t][P::NJ - 1]);
        }
#pragma unroll
        for (int v = 0; v < P::MV; ++v) {
            const Frag<BF> vf = col_rows<P::NJ>(T, P::LD, P::KW * kw, 16 * (wr * P::MV + v), lane);
#pragma unroll
            for (int t = 0; t < MT; ++t) O[t][v] = mma_rows<P::NJ>(vf, pf[t], O[t][v]);
        }
    }
    // join the key groups: common maximum, then the rescaled sums added to the first's, one after the other
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        l[t] = sum4g(l[t]);
        if (wr == 0 && g == 0) {
            Ms[kw * MT * 16 + 16 * t + r] = m[t];
            Ss[kw * MT * 16 + 16 * t + r] = l[t];
        }
    }
    lds_barrier();
    float ml[MT], sl[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        float mm = Ms[16 * t + r];
#pragma unroll
        for (int w = 1; w < P::WK; ++w) mm = fmaxf(mm, Ms[w * MT * 16 + 16 * t + r]);
        float sm = 0.f;
#pragma unroll
        for (int w = 0; w < P::WK; ++w) {
            // (an empty group counts for nothing; one of NaN scores has a NaN sum and no maximum)
            const float mw = Ms[w * MT * 16 + 16 * t + r], lw = Ss[w * MT * 16 + 16 * t + r];
            sm += lw == 0.f ? 0.f : lw * exp2_fast(mw - mm);
        }
        const float f = m[t] == -INFINITY ? 0.f : exp2_fast(m[t] - mm);
#pragma unroll
        for (int v = 0; v < P::MV; ++v) O[t][v] *= f;
        ml[t] = mm;
        sl[t] = sm;
    }
    // Every group ends with the sums of its own part of the columns: in round w it
    // hands the one w groups on its part and adds what it is handed.
    f32x4 *X = (f32x4 *)smem + lane;
#pragma unroll 1
    for (int w = 1; w < P::WK; ++w) {
        if (w > 1) lds_barrier(); // the previous round's readers are done
#pragma unroll
        for (int p = 0; p < P::WK; ++p) {
            if ((kw + w) % P::WK != p) continue;
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int v = 0; v < P::MP; ++v) X[(((wr * P::WK + p) * MT + t) * P::MP + v) * 64] = O[t][p * P::MP + v];
        }
        lds_barrier();
#pragma unroll
        for (int p = 0; p < P::WK; ++p) {
            if (kw != p) continue;
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int v = 0; v < P::MP; ++v) O[t][p * P::MP + v] += X[(((wr * P::WK + p) * MT + t) * P::MP + v) * 64];
        }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        const int i = row0 + 16 * t + r;
        if (i >= rows) continue;
        const size_t out = (size_t)nq * rows + i;
        const float inv = sl[t] != 0.f ? 1.f / sl[t] : 0.f;
#pragma unroll
        for (int v = 0; v < P::MV; ++v) {
            const int c = 16 * (wr * P::MV + v) + 4 * g;
            if (v / P::MP != kw || c >= a.dl) continue;
            if (slot >= 0) store4(a.part + ((size_t)slot * rows + i) * a.dl + c, O[t][v]);
            else store4((S *)a.o + out * a.dl + c, O[t][v] * inv);
        }
        if (wave == 0 && g == 0) {
            if (slot >= 0) {
                *reinterpret_cast<f32x2 *>(a.part_ml + ((size_t)slot * rows + i) * 2) = f32x2{ml[t], sl[t]};
            } else if (a.lse) {
                a.lse[out] = sl[t] == 0.f ? -INFINITY : (ml[t] + __builtin_amdgcn_logf(sl[t])) * 0.69314718055994531f;
            }
        }
    }
}

// PARTS: every piece is left as a part, at place unit + sequence (both only grow from
// one piece to the next, and one of them does)
template <bool BF, int DLP, int MT, bool PARTS = false>
__global__ __launch_bounds__(256, (DLP <= 128 && MT == 1 ? 3 : !BF && DLP == 256 ? 1 : 2)) void mla_step_kernel(MlaStepArgs a) {
    using P = StepShape<BF, DLP, MT>;
    using S = typename P::S;
    __shared__ __align__(16) unsigned char smem[P::TILE_B > P::MERGE_B ? P::TILE_B : P::MERGE_B];
    __shared__ __align__(16) S Qs[P::QL ? MT * 16 * P::LD : 8];
    __shared__ __align__(16) float bias[P::KT];
    __shared__ float Ms[P::WK * MT * 16], Ss[P::WK * MT * 16];
    const int lane = threadIdx.x & 63;
    const int rows = a.S * a.H, rb = (rows + MT * 16 - 1) / (MT * 16);
    // eight shares side by side on the eight XCDs, then the same shares' next
    // block of queries: it finds the rows in its XCD's L2
    const int blk = blockIdx.x / (8 * rb), in = blockIdx.x % (8 * rb);
    const int unit = blk * 8 + in % 8, row0 = (in / 8) * MT * 16;
    const Share sh = share_out(a, lane);
    const int from = unit * sh.share, to = min(from + sh.share, sh.total);
    if (unit >= a.units || from >= to) return;
    // the sequence the share begins in, and where that begins
    const int owner = __builtin_ctzll(__ballot(sh.before + sh.mine > from));
    int nq = owner * sh.per, begin = __builtin_amdgcn_readlane(sh.before, owner);
    for (int at = from; at < to;) {
        int tiles = seq_tiles(a, nq);
        while (begin + tiles <= at) {
            begin += tiles;
            tiles = seq_tiles(a, ++nq);
        }
        const int stop = min(begin + tiles, to);
        step_piece<BF, DLP, MT>(a, nq, (at - begin) << a.tile, (stop - begin) << a.tile, row0,
                                PARTS                                           ? unit + nq
                                : at == begin && stop == begin + tiles ? -1 : part_slot(unit, begin, sh.share),
                                smem, Qs, bias, Ms, Ss);
        at = stop;
    }
}
// Joins the parts of a sequence: o = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i.
// A workgroup takes one sequence's queries, `mine` at a time; four columns a
// thread, `groups` threads share the parts (part i with group i % groups, each
// in order, then the groups in order). Sequences one workgroup finished are
// done; empty ones get their zeros here.
template <bool BF> __global__ __launch_bounds__(256) void mla_join_kernel(MlaStepArgs a, int groups) {
    using S = typename Op<BF>::S;
    __shared__ __align__(16) f32x4 acc[256];
    __shared__ float ms[256], ls[256];
    const int cols = a.dl / 4, tid = threadIdx.x, rows = a.S * a.H;
    const int wide = min(cols, 256 / groups), per_row = wide * groups, mine = 256 / per_row;
    const int bpr = (rows + mine - 1) / mine, nq = blockIdx.x / bpr;
    const int q = tid / per_row, grp = tid % per_row / wide, c = (blockIdx.y * wide + tid % wide) * 4;
    const int i0 = blockIdx.x % bpr * mine + q;
    const Share sh = share_out(a, tid & 63);
    const int lane_of = nq / sh.per, tiles = seq_tiles(a, nq);
    int begin = __builtin_amdgcn_readlane(sh.before, lane_of);
    for (int n = lane_of * sh.per; n < nq; ++n) begin += seq_tiles(a, n);
    const int w0 = begin / sh.share, cnt = tiles ? (begin + tiles - 1) / sh.share - w0 + 1 : 0;
    if (cnt == 1) return;
    const bool on = q < mine && i0 < rows && c < a.dl;
    float m = -INFINITY, l = 0.f;
    f32x4 x = zero4();
    if (on) {
        // JB parts at a time, all requested before the first is used (past the last: that one again, with weight 0)
        constexpr int JB = 8;
        for (int p0 = grp; p0 < cnt; p0 += JB * groups) {
            f32x4 y[JB];
            f32x2 s[JB];
#pragma unroll
            for (int k = 0; k < JB; ++k) {
                const int p = min(p0 + k * groups, cnt - 1);
                const size_t at = (size_t)(p ? 2 * (w0 + p) : part_slot(w0, begin, sh.share)) * rows + i0;
                s[k] = *reinterpret_cast<const f32x2 *>(a.part_ml + at * 2);
                y[k] = *reinterpret_cast<const f32x4 *>(a.part + at * a.dl + c);
            }
            float mn = m;
#pragma unroll
            for (int k = 0; k < JB; ++k) mn = fmaxf(mn, s[k][0]);
            const float f = m == -INFINITY ? 0.f : exp2_fast(m - mn);
            x *= f;
            l *= f;
            m = mn;
#pragma unroll
            for (int k = 0; k < JB; ++k) {
                const float w = p0 + k * groups >= cnt || s[k][1] == 0.f ? 0.f : exp2_fast(s[k][0] - m);
                l = fmaf(w, s[k][1], l);
                x += (w != 0.f ? y[k] : zero4()) * w;
            }
        }
    }
    if (groups > 1) {
        acc[tid] = x;
        ms[tid] = m;
        ls[tid] = l;
        __syncthreads();
        if (grp != 0 || !on) return; // (threads left over have no parts, and none to read behind them)
        float mm = m;
        for (int k = 1; k < groups; ++k) mm = fmaxf(mm, ms[tid + k * wide]);
        f32x4 sum = zero4();
        float sl = 0.f;
        for (int k = 0; k < groups; ++k) {
            const float lk = ls[tid + k * wide], w = lk == 0.f ? 0.f : exp2_fast(ms[tid + k * wide] - mm);
            sl = fmaf(w, lk, sl);
            if (w != 0.f) sum += acc[tid + k * wide] * w;
        }
        x = sum;
        l = sl;
        m = mm;
    }
    if (!on) return;
    const size_t row = (size_t)nq * rows + i0;
    store4((S *)a.o + row * a.dl + c, x * (l != 0.f ? 1.f / l : 0.f));
    if (a.lse && c == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f;
}

int step_class(int dl) {
    return dl <= 64 ? 64 : dl <= 128 ? 128 : dl <= 192 ? 192 : dl <= 256 ? 256 : dl <= 384 ? 384 : 512;
}

// workgroups a CU holds at once, by their registers and LDS
static int step_per_cu(const MlaStepArgs &a, bool bf16) {
    const int c = step_class(a.dl);
    if (bf16) return c == 64 ? 5 - a.mt : c == 128 ? 4 - a.mt : 2;
    return c == 64 ? 3 : c == 128 ? 2 : 1;
}

void mla_step_plan(MlaStepArgs &a, bool bf16, int cus) {
    const long long rows = (long long)a.S * a.H, cap = (long long)a.cols * a.page;
    a.tile = step_tile(step_class(a.dl));
    const long long most = a.N * ((cap + (1 << a.tile) - 1) >> a.tile); // tiles there may be
    // Query blocks per workgroup: two where the registers hold them and there may
    // be twelve tiles for each CU, which pays for a longer start and end (fp32,
    // 24 queries of 256 + 64, 48 sequences up to 1500 rows: 48 us with two, 42
    // with one; up to 6000: 96 and 103); at 64 columns a block's rows cost too
    // little to be shared (32 queries, 200 sequences up to 2000: 31 and 29 us).
    a.mt = rows > 16 && a.dl > 64 && a.dl <= 256 && most >= 12LL * cus ? 2 : 1;
    const long long rb = (rows + 16 * a.mt - 1) / (16 * a.mt);
    // as many shares as the chip holds, each a tile or more
    long long n = (long long)cus * step_per_cu(a, bf16) / rb;
    if (n > most) n = most;
    a.units = n < 1 ? 1 : (int)n;
}

static long long step_grid(const MlaStepArgs &a) { // (eight shares side by side, see the kernel)
    return ((long long)a.units + 7) / 8 * 8 * (((long long)a.S * a.H + 16 * a.mt - 1) / (16 * a.mt));
}
template <bool BF, int DLP, int MT, bool PARTS> static hipError_t step_run(const MlaStepArgs &a, hipStream_t st) {
    hipLaunchKernelGGL((mla_step_kernel<BF, DLP, MT, PARTS>), dim3((unsigned)step_grid(a)), dim3(256), 0, st, a);
    return hipGetLastError();
}
template <bool BF, int DLP, bool PARTS> static hipError_t step_rows(const MlaStepArgs &a, hipStream_t st) {
    if constexpr (DLP > 64 && DLP <= 256)
        if (a.mt == 2) return step_run<BF, DLP, 2, PARTS>(a, st);
    return step_run<BF, DLP, 1, PARTS>(a, st);
}
template <bool BF, bool PARTS> static hipError_t step_launch(const MlaStepArgs &a, hipStream_t st) {
    switch (step_class(a.dl)) {
    case 64: return step_rows<BF, 64, PARTS>(a, st);
    case 128: return step_rows<BF, 128, PARTS>(a, st);
    case 192: return step_rows<BF, 192, PARTS>(a, st);
    case 256: return step_rows<BF, 256, PARTS>(a, st);
    case 384: return step_rows<BF, 384, PARTS>(a, st);
    default: return step_rows<BF, 512, PARTS>(a, st);
    }
}
hipError_t launch_mla_step(const MlaStepArgs &a, bool bf16, hipStream_t st) {
    return bf16 ? step_launch<true, false>(a, st) : step_launch<false, false>(a, st);
}
hipError_t launch_mla_step_parts(const MlaStepArgs &a, bool bf16, hipStream_t st) {
    return bf16 ? step_launch<true, true>(a, st) : step_launch<false, true>(a, st);
}

// Launch of the join. The parts of an average sequence decide how many threads share them.
struct JoinGrid {
    int groups, wide;
    long long x;
};
static JoinGrid join_grid(const MlaStepArgs &a) {
    int groups = 1;
    while (groups < 16 && groups * 8LL * a.N < a.units) groups *= 2;
    const int cols = a.dl / 4, wide = cols < 256 / groups ? cols : 256 / groups, mine = 256 / (wide * groups);
    return {groups, wide, a.N * (((long long)a.S * a.H + mine - 1) / mine)};
}
long long mla_step_groups(const MlaStepArgs &a) {
    if (a.units == 0) return 0;
    const long long x = step_grid(a), y = join_grid(a).x;
    return x > y ? x : y;
}

hipError_t launch_mla_join(const MlaStepArgs &a, bool bf16, hipStream_t st) {
    const JoinGrid j = join_grid(a);
    const int groups = j.groups, cols = a.dl / 4;
    const dim3 grid((unsigned)j.x, (unsigned)((cols + j.wide - 1) / j.wide));
    if (bf16) hipLaunchKernelGGL(mla_join_kernel<true>, grid, dim3(256), 0, st, a, groups);
    else hipLaunchKernelGGL(mla_join_kernel<false>, grid, dim3(256), 0, st, a, groups);
    return hipGetLastError();
}

} // namespace gdn
