// Shared prefixes: the bf16 instances, how a call is shared out, and the join.
#include "gdn_mla_prefix.hpp"

namespace gdn {

template <int DLP, int KS> static hipError_t rows_bf16(const PrefixArgs &a, hipStream_t st) {
    if constexpr (DLP > 192) return prefix_run<true, DLP, KS, 1>(a, st);
    else return a.qt == 2 ? prefix_run<true, DLP, KS, 2>(a, st) : prefix_run<true, DLP, KS, 1>(a, st);
}
// (a rotary part of 32 columns or less needs one step of the product less)
template <int DLP> static hipError_t steps_bf16(const PrefixArgs &a, hipStream_t st) {
    return a.dl + a.dr <= DLP + 32 ? rows_bf16<DLP, DLP / 32 + 1>(a, st) : rows_bf16<DLP, DLP / 32 + 2>(a, st);
}
hipError_t launch_mla_prefix_bf16(const PrefixArgs &a, hipStream_t st) {
    switch (step_class(a.dl)) {
    case 64: return steps_bf16<64>(a, st);
    case 128: return steps_bf16<128>(a, st);
    case 192: return steps_bf16<192>(a, st);
    case 256: return steps_bf16<256>(a, st);
    case 384: return steps_bf16<384>(a, st);
    default: return steps_bf16<512>(a, st);
    }
}

long long mla_prefix_blocks(const PrefixArgs &a) {
    const long long rows = (long long)a.N * a.S * a.H;
    return rows / a.qb + (a.G < a.N ? a.G : a.N); // (every group may leave its last block unfilled)
}
void mla_prefix_plan(PrefixArgs &a, bool bf16, int cus) {
    const int c = step_class(a.dl);
    // Two blocks of queries a wave where a group fills them: each tile read from LDS then serves twice as many products
    // (256 sequences, 16 heads, behind one prefix of 8192 rows: 64 columns 41 us with one, 37 with two, 128: 51 and 48, 192:
    // 67 and 61; 256, where two spill, 75 and 130; eight groups of 96 queries, 128 columns: 21 and 22).
    a.qt = bf16 && c <= 192 && (long long)a.N * a.S * a.H >= 256LL * (a.G < a.N ? a.G : a.N) ? 2 : 1;
    a.qb = 16 * prefix_nw(bf16, c) * a.qt;
    a.units = cus * prefix_per_cu(bf16, c);
    // the walks may hold so many tiles
    const int kt = prefix_tile(bf16, c);
    const long long rows = (long long)a.S * a.H, cap = ((long long)a.cols * a.page + kt - 1) / kt + PREFIX_START;
    const long long own_cap = ((long long)a.own_cols * a.page + kt - 1) / kt + PREFIX_START;
    a.own_blocks = (int)((rows + a.qb - 1) / a.qb);
    a.own_qb = (int)(rows < a.qb ? rows : a.qb);
    long long most = mla_prefix_blocks(a) * cap;
    // Own rows are walked here as well, which saves a launch and its starts (48 sequences of three drafts and 700 rows
    // of 512 + 64: 105 us with a launch of their own, 88 without; 256 sequences of 1024 rows of 128 + 32: 79 and 76; five
    // short ones in fp32: 21 and 18), though a sequence's queries leave waves idle: in bf16, where the rows' bytes take
    // the time even so. In fp32 the products do: there if they fill the waves, or if all walks may not fill the chip.
    // (Lengths are known on the GPU alone. Where own rows are nearly all there is, 4096 of them behind a prefix of 64, 16
    // queries, this kernel takes 93 us for 256 sequences of 128 + 32 and 78 for 48 of 512 + 64, the step's alone 70 and 49;
    // with 48 queries a sequence 97 and 104.)
    a.own = bf16 || 4 * rows >= 3LL * a.qb || most + a.N * a.own_blocks * own_cap <= a.units;
    if (a.own) most += a.N * a.own_blocks * own_cap;
    if (most < a.units) a.units = (int)most;
}

// The parts of a query: its own rows' and its prefix's, added up relative to
// the largest maximum among them. A thread takes four columns of a query, eight parts requested at
// a time.
template <bool BF> __global__ __launch_bounds__(256) void mla_shared_join_kernel(MlaStepArgs a, PrefixArgs p, int kt) {
    using S = typename Op<BF>::S;
    const int cols = a.dl / 4, tid = threadIdx.x, lane = tid & 63, rows = a.S * a.H;
    const int mine = 256 / cols, bpr = (rows + mine - 1) / mine, nq = blockIdx.x / bpr;
    const int q = tid / cols, c = tid % cols * 4, i0 = blockIdx.x % bpr * mine + q;
    const Line s = line_of(p, lane, kt);
    // own rows
    int own, own_slot, own_qb, own_in;
    long long share;
    if (p.own) { // (a token that is no padding has rows, so its sequence's walk was noted)
        const int tiles = tiles_of(p, p.G + nq, kt), block = i0 / p.qb;
        const long long at = p.walks[2 * nq] + (long long)block * walk_of(tiles) + PREFIX_START;
        share = max(p.walks[2 * nq + 1], 1LL);
        own_slot = (int)(at / share);
        own = tiles ? (int)((at + tiles - 1) / share) - own_slot + 1 : 0;
        own_slot += nq * p.own_blocks + block;
        own_qb = p.own_qb;
        own_in = i0 - block * p.qb;
    } else {
        share = share_of(p, s.total);
        const Share sh = share_out(a, lane);
        const int lane_of = nq / sh.per, tiles = seq_tiles(a, nq);
        int begin = __builtin_amdgcn_readlane(sh.before, lane_of);
        for (int n = lane_of * sh.per; n < nq; ++n) begin += seq_tiles(a, n);
        const int w0 = begin / sh.share;
        own = tiles ? (begin + tiles - 1) / sh.share - w0 + 1 : 0;
        own_slot = w0 + nq;
        own_qb = rows;
        own_in = i0;
    }
    // the prefix: the group of this sequence, if any
    long long at0 = 0; // the walks before the first block of the group
    int block0 = 0, first = 0, ptiles = 0, pwalk = 0;
    {
        int most = s.most, end = 0;
        for (int i = 0; i < s.per; ++i) {
            if (lane * s.per + i >= p.G) break;
            end = group_of(p, lane * s.per + i, most, kt).hi;
        }
        const uint64_t past = __ballot(end > nq);
        if (past) {
            const int l = __builtin_ctzll(past);
            most = __shfl(s.most, l, 64);
            block0 = __shfl(s.blocks0, l, 64);
            at0 = __shfl(s.tiles0, l, 64);
            for (int i = 0; i < s.per; ++i) {
                const Group x = group_of(p, l * s.per + i, most, kt);
                if (nq < x.hi) {
                    if (nq >= x.lo) {
                        first = x.lo;
                        ptiles = x.tiles;
                        pwalk = x.walk;
                    }
                    break;
                }
                block0 += x.blocks;
                at0 += (long long)x.blocks * x.walk;
            }
        }
    }
    if (q >= mine || i0 >= rows) return;
    const size_t row = (size_t)nq * rows + i0;
    const int qb = p.qb, in = (nq - first) * rows + i0, block = in / qb;
    const long long pb = at0 + (long long)block * pwalk + PREFIX_START;
    const int u0 = ptiles ? (int)(pb / share) : 0, parts = ptiles ? (int)((pb + ptiles - 1) / share) - u0 + 1 : 0;
    const bool real = seq_rows(a, nq) - a.S + i0 / a.H >= 0; // (a token before position 0 is padding)
    float m = -INFINITY, l = 0.f;
    f32x4 x = zero4();
    if (real) {
        constexpr int JB = 8;
        for (int k0 = 0; k0 < own + parts; k0 += JB) {
            f32x4 y[JB];
            f32x2 st[JB];
#pragma unroll
            for (int k = 0; k < JB; ++k) { // (past the last: that one again, with weight 0)
                const int j = min(k0 + k, own + parts - 1);
                const size_t at = j < own ? (size_t)(own_slot + j) * own_qb + own_in
                                          : (size_t)(u0 + (j - own) + block0 + block) * qb + (in - block * qb);
                st[k] = *reinterpret_cast<const f32x2 *>((j < own ? p.own_part_ml : p.part_ml) + at * 2);
                y[k] = *reinterpret_cast<const f32x4 *>((j < own ? p.own_part : p.part) + at * a.dl + c);
            }
            float mn = m;
#pragma unroll
            for (int k = 0; k < JB; ++k) mn = fmaxf(mn, st[k][0]);
            const float f = m == -INFINITY ? 0.f : exp2_fast(m - mn);
            x *= f;
            l *= f;
            m = mn;
#pragma unroll
            for (int k = 0; k < JB; ++k) {
                const float w = k0 + k >= own + parts || st[k][1] == 0.f ? 0.f : exp2_fast(st[k][0] - m);
                l = fmaf(w, st[k][1], l);
                x += (w != 0.f ? y[k] : zero4()) * w;
            }
        }
    }
    store4((S *)a.o + row * a.dl + c, x * (l != 0.f ? 1.f / l : 0.f));
    if (a.lse && c == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * 0.69314718055994531f;
}

long long mla_shared_join_groups(const MlaStepArgs &a) {
    const int mine = 256 / (a.dl / 4);
    return a.N * (((long long)a.S * a.H + mine - 1) / mine);
}
hipError_t launch_mla_shared_join(const MlaStepArgs &a, const PrefixArgs &p, bool bf16, hipStream_t st) {
    const dim3 grid((unsigned)mla_shared_join_groups(a));
    const int kt = prefix_tile(bf16, step_class(a.dl));
    if (bf16) hipLaunchKernelGGL(mla_shared_join_kernel<true>, grid, dim3(256), 0, st, a, p, kt);
    else hipLaunchKernelGGL(mla_shared_join_kernel<false>, grid, dim3(256), 0, st, a, p, kt);
    return hipGetLastError();
}

} // namespace gdn
