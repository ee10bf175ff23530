// Attention of a serving batch against prefixes that groups of its sequences
// share, and against the sequences' own rows beside them.
//
//   z_j = scale q . row_j,  o = sum_j softmax(z)_j row_j[:dl] over the prefix's rows and the own ones
//
// A prefix's rows are seen by every query of its group, thousands of them, so
// this is a matrix product as in the attention of a prompt, without a mask: S^T =
// K Q^T and O^T = V^T P^T over tiles of cached rows in LDS, a lane owning one
// query, the probabilities at once the operand of the second product, V read from the same tile by transposing
// reads. (In bf16 they are rounded to it, as in the step: against 64 bits o is off by 0.0017 to 0.0020 of its size
// where 32-bit probabilities leave the 0.0017 of its own rounding; two operands for their two halves would be half as
// many products again.) A
// wave takes 16 * QT queries of a group, which stay in registers; the waves of a
// workgroup walk tiles of rows that they share, two tiles in LDS, the next one
// requested before this one is used, straight from memory (through registers a
// wide latent spills hundreds of them: 407 us for 72).
// A sequence's own rows are a group of its own behind the prefixes', masked in
// the last tile.
// The walks of all blocks of queries, end to end, are cut into equal shares,
// one for each workgroup the chip holds, whatever the groups' sizes and
// lengths. Every piece leaves its sums as a part, at place (share + block): both
// only grow from one piece to the next, and one of them does. The join adds up a query's parts.
//
// Measured: 256 sequences of up to 1024 rows behind a prefix of 16384, 16 heads of 128 + 32
// bf16: 71 us and 10 us for the join; 48 sequences of three drafts, four prefixes of 4096 to 8191
// rows, 512 + 64 bf16: 78 and 15 us. No unit is half busy (matrix products 23 and 19 % of the time,
// vector instructions 29 and 17, LDS 18 and 23, which reads 256 bytes a cycle): of the waves' time
// 41 and 42 % go by in waits for a tile or an operand, 25 and 32 % in waits to issue. A SIMD's two
// waves go through scores, exponentials and values between the same barriers. 512 columns: a wave
// reads all of a tile for 16 queries, which is what its registers hold beside their sums; the parts'
// 61 MB are written and read again. (Loads of a tile took as many vector instructions again before
// rows' addresses went through the wave and the walk lost its divisions.)
#pragma once

#include "gdn_lds_tile.hpp"
#include "gdn_serve.hpp"

namespace gdn {

constexpr float PREFIX_RAISE = 8.f; // lazy maximum, as in the forward over expanded heads

// Waves of a workgroup, and rows of a tile, by the padded latent columns: beyond 256 the
// operands of 16 queries fill what two waves per SIMD have of registers, so
// eight waves share a tile (what one wave per SIMD would hold for 32 the compiler spills).
__host__ __device__ constexpr int prefix_nw(bool bf, int dlp) { return bf && dlp > 256 ? 8 : 4; }
__host__ __device__ constexpr int prefix_tile(bool bf, int dlp) { return bf && (dlp <= 128 || dlp > 256) ? 64 : 32; }
template <bool BF, int DLP, int KS, int QT> struct PrefixShape {
    using S = typename Op<BF>::S;
    using Tile = LdsTile<BF, KS>;
    static constexpr int NW = prefix_nw(BF, DLP), NT = 64 * NW, V = Tile::V, RU = Tile::RU, XM = Tile::XM, MV = DLP / 16,
                         QB = 16 * NW * QT, KT = prefix_tile(BF, DLP), TILE = KT * RU, // (units)
                         NL = TILE / NT; // loads of a thread
    static_assert(TILE % NT == 0 && KT % NW == 0, "every load moves 64 units of a wave's rows");
};

__device__ const u32x4 prefix_zeros[576 * 4 / 16] = {}; // a row of them

// A walk's start (the first tile's wait, the queries) counts as so many tiles.
constexpr int PREFIX_START = 2;

// The groups' walks, end to end: lane l holds groups l * per .. + per - 1. Where the sequences' own
// rows are walked here too, those walks follow, each sequence as a group of its own.
struct Line {
    int per, most;           // groups per lane; largest start before this lane's
    int blocks0, blocks;     // blocks of queries before this lane's, in them
    long long tiles0, tiles; // their walks' lengths
    long long total;         // length of all groups' walks
};
struct Group {
    int lo, hi;                    // its sequences
    int rows, blocks, tiles, walk; // its queries, their blocks, the tiles of its rows, the length of a block's walk
};
__device__ __forceinline__ int prefix_rows(const PrefixArgs &a, int g) { // g >= G: own rows of sequence g - G
    return g < a.G ? (int)min((long long)max(a.plens[g], 0), (long long)a.cols * a.page)
                   : (int)min((long long)max(a.lens[g - a.G], 0), (long long)a.own_cols * a.page);
}
__device__ __forceinline__ int tiles_of(const PrefixArgs &a, int g, int kt) {
    return (int)(((long long)prefix_rows(a, g) + kt - 1) / kt);
}
__device__ __forceinline__ int walk_of(int tiles) { return tiles ? tiles + PREFIX_START : 0; }
// a workgroup's share (a tile at least: where the chip is not full, the longest walk is the call's time, and the
// parts are few; two prefixes of 700 rows of 64 + 16 in fp32: 15 us with four tiles, 11 with two, 8 with one)
__device__ __forceinline__ long long share_of(const PrefixArgs &a, long long total) {
    return max((total + a.units - 1) / a.units, 1LL);
}
__device__ __forceinline__ int start_of(const PrefixArgs &a, int g) { return min(max(a.starts[g], 0), a.N); }
// most: the largest start before (starts that go back count as that)
__device__ __forceinline__ Group group_of(const PrefixArgs &a, int g, int &most, int kt) {
    Group x;
    x.lo = max(most, start_of(a, g));
    x.hi = max(x.lo, start_of(a, g + 1));
    most = x.lo;
    x.rows = (x.hi - x.lo) * a.S * a.H;
    x.blocks = (x.rows + a.qb - 1) / a.qb;
    x.tiles = tiles_of(a, g, kt);
    x.walk = walk_of(x.tiles);
    return x;
}
__device__ __forceinline__ Line line_of(const PrefixArgs &a, int lane, int kt) {
    Line s;
    s.per = (a.G + 63) / 64;
    int m = 0;
    for (int i = 0; i < s.per; ++i)
        if (lane * s.per + i < a.G) m = max(m, start_of(a, lane * s.per + i));
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(m, o, 64);
        if (lane >= o) m = max(m, y);
    }
    const int up = __shfl_up(m, 1, 64);
    s.most = lane ? up : 0;
    s.blocks = 0;
    s.tiles = 0;
    int most = s.most;
    for (int i = 0; i < s.per; ++i) {
        if (lane * s.per + i >= a.G) break;
        const Group x = group_of(a, lane * s.per + i, most, kt);
        s.blocks += x.blocks;
        s.tiles += (long long)x.blocks * x.walk;
    }
    int b = s.blocks;
    long long t = s.tiles;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int y = __shfl_up(b, o, 64);
        const long long z = __shfl_up(t, o, 64);
        if (lane >= o) {
            b += y;
            t += z;
        }
    }
    s.blocks0 = b - s.blocks;
    s.tiles0 = t - s.tiles;
    s.total = __shfl(t, 63, 64);
    return s;
}

// Tiles [t0, t1) of group g's rows for the queries row0 .. of its `rows`; the sums go to part `slot`.
template <bool BF, int DLP, int KS, int QT>
__device__ __forceinline__ void prefix_piece(const PrefixArgs a, int g, int lo, int rows, int row0, int t0, int t1,
                                             int slot, u32x4 *T0, float *bias0) {
    using P = PrefixShape<BF, DLP, KS, QT>;
    using S = typename P::S;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), r = lane & 15,
              gr = lane >> 4;
    const int d = a.dl + a.dr, n = prefix_rows(a, g);
    // Tile row `lane`: its column of the table and its place in that page, of the tile asked for next; the table entry
    // is requested two tiles ahead, and where the row is known one ahead (none: among zeros).
    const bool own = g >= a.G;
    const int *tb = own ? a.own_table + (size_t)(g - a.G) * a.own_cols : a.table + (size_t)g * a.cols;
    const int over = P::KT % a.page, across = P::KT / a.page;
    int col = (t0 * P::KT + lane) / a.page, in = t0 * P::KT + lane - col * a.page, entry = -1;
    uint64_t row = 0;
    bool some = false;
    auto ask = [&](int tile) {
        if (lane < P::KT && tile * P::KT + lane < n) entry = tb[col];
    };
    auto place = [&](int tile) {
        some = lane < P::KT && tile * P::KT + lane < n && (unsigned)entry < (unsigned)a.pages;
        const S *at = (const S *)a.cache + (uint64_t)((unsigned)entry * (unsigned)a.page + (unsigned)in) * (unsigned)d;
        row = some ? (uint64_t)at : (uint64_t)&prefix_zeros;
        in += over;
        col += across;
        if (in >= a.page) {
            in -= a.page;
            ++col;
        }
    };
    // A tile goes from memory to LDS without passing registers: a wave's load
    // takes 64 units that follow each other in LDS, each lane's from where it stands in its
    // row. Units past the row's end are not loaded (the kernel cleared them). A lane's row and unit are formed anew for each
    // tile where registers are short.
    const uint32_t T1 = lds_place(T0 + wave * P::NL * 64);
    const int row_units = d / P::V;
    auto fetch = [&](int buf) {
        int jj = lane;
        if constexpr (DLP > 128) asm volatile("" : "+v"(jj));
        int u = jj % P::RU;
        jj /= P::RU;
#pragma unroll
        for (int i = 0; i < P::NL; ++i) {
            const int j = wave * (P::KT / P::NW) + jj, at = u ^ (j & P::XM);
            const uint32_t lo = __builtin_amdgcn_ds_bpermute(4 * j, (int)(uint32_t)row),
                           hi = __builtin_amdgcn_ds_bpermute(4 * j, (int)(uint32_t)(row >> 32));
            if (at < row_units)
                load_to_lds((const char *)((uint64_t)hi << 32 | lo) + 16 * (unsigned)at, T1 + (buf * P::TILE + i * 64) * 16);
            jj += 64 / P::RU;
            u += 64 % P::RU;
            if (u >= P::RU) {
                u -= P::RU;
                ++jj;
            }
            if (DLP > 128 && i % 2) in_flight(); // (all requested at once would spill)
        }
        if (wave == 0 && lane < P::KT) bias0[buf * P::KT + lane] = some ? 0.f : -INFINITY;
    };
    lds_barrier(); // (the previous piece's readers are done)
    ask(t0);
    place(t0);
    fetch(0);
    if (t0 + 1 < t1) ask(t0 + 1);
    Frag<BF> Q[QT][KS];
    const S *qp = (const S *)a.q + ((size_t)lo * a.S * a.H) * d;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int i = row0 + (wave * QT + t) * 16 + r;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
            const int c = 32 * k + 8 * gr;
            Q[t][k] = row8_if(i < rows && c < d, qp + (size_t)i * d + c);
        }
    }
    // Own rows are seen up to the token's own: rows below `see`, which the tiles before the last tokens' need not ask.
    int see[QT];
#pragma unroll
    for (int t = 0; t < QT; ++t) see[t] = own ? n - a.S + 1 + (row0 + (wave * QT + t) * 16 + r) / a.H : 2147483647;
    const int all_see = own ? n - a.S + 1 : 2147483647;
    const bool idle = row0 + wave * QT * 16 >= rows; // (a wave without queries only helps with the loads)
    f32x4 O[QT][P::MV];
    float m[QT], l[QT];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        m[t] = -INFINITY;
        l[t] = 0.f;
#pragma unroll
        for (int v = 0; v < P::MV; ++v) O[t][v] = zero4();
    }
    const float c2 = a.scale * (float)LOG2E;
    TileReads<typename P::Tile> at;
    at.init(lane);
    wait_vmem(); // the first tile, and the queries
    lds_barrier();
    for (int tile = t0; tile < t1; ++tile) {
        const int buf = (tile - t0) & 1;
        const u32x4 *T = T0 + buf * P::TILE;
        const float *bias = bias0 + buf * P::KT;
        if (tile + 1 < t1) {
            place(tile + 1);
            fetch(buf ^ 1); // (its last readers passed the barrier before this tile)
            if (tile + 2 < t1) ask(tile + 2);
        }
#pragma unroll 1
        for (int u = idle ? P::KT / 32 : 0; u < P::KT / 32; ++u) {
            // absent rows: scores of -inf from the start (their keys are zero)
            f32x4 X[QT][2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const f32x4 bj = *reinterpret_cast<const f32x4 *>(bias + 32 * u + 16 * j + 4 * gr);
#pragma unroll
                for (int t = 0; t < QT; ++t) X[t][j] = bj;
            }
            // Operands are requested a group ahead of the products that take them, and no further: left
            // to itself the compiler requests all of them at once and spills what it holds.
            constexpr int KG = BF && DLP <= 256 ? 2 : 1, NK = (KS + KG - 1) / KG, VG = 2 * KG, NV = P::MV / VG;
            Frag<BF> kf[2][KG][2], vf[2][VG];
            auto keys = [&](int i) {
#pragma unroll
                for (int k = 0; k < KG; ++k)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        if (i * KG + k < KS) kf[i & 1][k][j] = at.rows(T, 32 * u + 16 * j, i * KG + k);
            };
            auto values = [&](int i) {
#pragma unroll
                for (int v = 0; v < VG; ++v) vf[i & 1][v] = at.cols(T, 32 * u, i * VG + v);
            };
            keys(0);
#pragma unroll
            for (int i = 0; i < NK; ++i) {
                if (i + 1 < NK) keys(i + 1);
                else values(0);
                in_flight();
#pragma unroll
                for (int k = 0; k < KG; ++k)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int t = 0; t < QT; ++t)
                            if (i * KG + k < KS) X[t][j] = mma8(kf[i & 1][k][j], Q[t][i * KG + k], X[t][j]);
                in_flight();
            }
            // What a token does not see is taken out behind the product, whatever its rows' scores came to. (In the
            // product with the values such a row still has its place, with probability 0: finite values leave no
            // trace, a NaN or infinity reaches the sequence's other tokens, as in the step.) The products'
            // results are waited for by hand: the compiler, ROCm 7.2, leaves the wait out behind a conditional block.
            if constexpr (QT == 2) asm volatile("s_nop 15" : "+v"(X[0][0]), "+v"(X[0][1]), "+v"(X[1][0]), "+v"(X[1][1]));
            else asm volatile("s_nop 15" : "+v"(X[0][0]), "+v"(X[0][1]));
            const int from = tile * P::KT + 32 * u;
            if (from + 32 > all_see) {
#pragma unroll
                for (int t = 0; t < QT; ++t)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (from + 16 * j + 4 * gr + e >= see[t]) X[t][j][e] = -INFINITY;
            }
            bool raise = false;
            float mx[QT];
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                float x = X[t][0][0];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x = fmaxf(x, X[t][j][e]);
                mx[t] = x * c2;
                raise |= mx[t] > m[t] + PREFIX_RAISE;
            }
            if (__any(raise)) {
#pragma unroll
                for (int t = 0; t < QT; ++t) {
                    const float mn = fmaxf(m[t], max4g(mx[t]));
                    const float f = mn == -INFINITY ? 1.f : exp2_fast(m[t] - mn);
                    m[t] = mn;
                    l[t] *= f;
#pragma unroll
                    for (int v = 0; v < P::MV; ++v) {
                        O[t][v] *= f;
                        if (v % 4 == 3) in_flight();
                    }
                }
            }
            Frag<BF> pf[QT];
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                const float mt = m[t] == -INFINITY ? 0.f : m[t];
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) X[t][j][e] = exp2_fast(fmaf(X[t][j][e], c2, -mt));
                const f32x4 sum = X[t][0] + X[t][1];
                l[t] += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                pf[t] = acc8<BF>(X[t][0], X[t][1]);
            }
            in_flight();
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (i + 1 < NV) values(i + 1);
                in_flight();
#pragma unroll
                for (int v = 0; v < VG; ++v)
#pragma unroll
                    for (int t = 0; t < QT; ++t) O[t][i * VG + v] = mma8(vf[i & 1][v], pf[t], O[t][i * VG + v]);
                in_flight();
            }
        }
        wait_vmem(); // the next tile is in LDS
        lds_barrier();
    }
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int i = (wave * QT + t) * 16 + r;
        const float sum = sum4g(l[t]);
        if (row0 + i >= rows) continue;
        const size_t to = (size_t)slot * (own ? a.own_qb : P::QB) + i;
        float *part = own ? a.own_part : a.part, *part_ml = own ? a.own_part_ml : a.part_ml;
#pragma unroll
        for (int v = 0; v < P::MV; ++v) {
            const int c = 16 * v + 4 * gr;
            if (c < a.dl) store4(part + to * a.dl + c, O[t][v]);
        }
        if (gr == 0) *reinterpret_cast<f32x2 *>(part_ml + to * 2) = f32x2{m[t], sum};
    }
}

// workgroups a CU holds, by registers and LDS
__host__ __device__ constexpr int prefix_per_cu(bool bf, int dlp) { return bf ? dlp <= 256 ? 2 : 1 : dlp <= 128 ? 2 : 1; }

// a value that is the same in all lanes, as one that needs no vector register
__device__ __forceinline__ int one(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ long long one(long long x) {
    return (long long)(((uint64_t)(uint32_t)one((int)(x >> 32)) << 32) | (uint32_t)one((int)x));
}

template <bool BF, int DLP, int KS, int QT>
__global__ __launch_bounds__(64 * prefix_nw(BF, DLP), prefix_per_cu(BF, DLP) * prefix_nw(BF, DLP) / 4) void mla_prefix_kernel(PrefixArgs a) {
    using P = PrefixShape<BF, DLP, KS, QT>;
    __shared__ u32x4 T[2 * P::TILE];
    __shared__ __align__(16) float bias[2 * P::KT];
    const int lane = threadIdx.x & 63, unit = blockIdx.x;
    if ((a.dl + a.dr) / P::V < P::RU) // units that no row fills
        for (int i = threadIdx.x; i < 2 * P::TILE; i += P::NT) T[i] = u32x4{0u, 0u, 0u, 0u};
    const Line s = line_of(a, lane, P::KT);
    Pieces own = {};
    auto walks = [&](int n) { return walk_of(tiles_of(a, a.G + n, P::KT)); };
    if (a.own) own = Pieces::of(a.N, walks, lane);
    const long long groups = one(s.total), all = groups + (long long)one(own.total) * a.own_blocks;
    const long long share = one(share_of(a, all)), from = unit * share, to = min(from + share, all);
    if (from >= to) return;
    auto own_group = [&](int n) {
        const int tiles = tiles_of(a, a.G + n, P::KT);
        return Group{n, n + 1, a.S * a.H, a.own_blocks, tiles, walk_of(tiles)};
    };
    // the group, or the sequence's own rows, that the share begins in
    int g, most = 0, block0 = 0;
    long long begin;
    Group x;
    if (from < groups) {
        const int owner = __builtin_ctzll(__ballot(s.tiles0 + s.tiles > from));
        g = owner * s.per;
        most = one(__shfl(s.most, owner, 64));
        block0 = one(__shfl(s.blocks0, owner, 64));
        begin = one(__shfl(s.tiles0, owner, 64));
        x = group_of(a, g, most, P::KT);
    } else { // (each of a sequence's blocks has a walk: found by their number)
        int n, in;
        const int number = (int)((from - groups) / a.own_blocks);
        own.find(walks, number, lane, n, in);
        n = one(n);
        g = a.G + n;
        begin = groups + (long long)(number - one(in)) * a.own_blocks;
        x = own_group(n);
    }
    for (long long at = from; at < to;) {
        while (begin + (long long)x.blocks * x.walk <= at) {
            begin += (long long)x.blocks * x.walk;
            block0 += x.blocks;
            ++g;
            x = g < a.G ? group_of(a, g, most, P::KT) : own_group(g - a.G);
        }
        if (g >= a.G && at == begin && threadIdx.x == 0) { // (for the join)
            a.walks[2 * x.lo] = begin;
            a.walks[2 * x.lo + 1] = share;
        }
        const int block = (int)((at - begin) / x.walk);
        const long long first = begin + (long long)block * x.walk, stop = min(first + x.walk, to);
        const int t0 = max((int)(at - first) - PREFIX_START, 0), t1 = (int)(stop - first) - PREFIX_START;
        if (t0 < t1)
            prefix_piece<BF, DLP, KS, QT>(a, g, x.lo, x.rows, block * P::QB, t0, t1,
                                          unit + block + (g < a.G ? block0 : x.lo * a.own_blocks), T, bias);
        at = stop;
    }
}

template <bool BF, int DLP, int KS, int QT> hipError_t prefix_run(const PrefixArgs &a, hipStream_t st) {
    hipLaunchKernelGGL((mla_prefix_kernel<BF, DLP, KS, QT>), dim3((unsigned)a.units), dim3(64 * prefix_nw(BF, DLP)), 0, st, a);
    return hipGetLastError();
}

} // namespace gdn
