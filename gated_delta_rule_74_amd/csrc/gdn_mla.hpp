// Latent attention and the paged latent cache: argument blocks, launch
// interface and device building blocks shared by their kernels (gfx950).
#pragma once

#include "gdn_common.hpp"
#include "gdn_launch.hpp"

namespace gdn {

// bracketed(): runs `launch`, between two of the caller's timing events while
// gdn_time_launches has them on (kinds as listed at gdn_launch_kind).
enum MlaKind {
    K_MLA_FWD = 8,
    K_MLA_BWD_Q,
    K_MLA_BWD_K,
    K_MLA_ROPE_SUM,
    K_MLA_STEP,
    K_MLA_JOIN,
    K_NORM_ROPE,
    K_NORM_ROPE_BWD,
    K_NORM_SUM,
    K_MLA_WRITE,
    K_PAGE_PLAN,
    K_PAGE_FILL
};
hipError_t bracket_begin(int kind, hipStream_t st);
hipError_t bracket_end(hipStream_t st);
template <class F> hipError_t bracketed(int kind, F &&launch, hipStream_t st) {
    hipError_t e = bracket_begin(kind, st);
    if (e == hipSuccess) e = launch();
    return e == hipSuccess ? bracket_end(st) : e;
}

// Expanded heads: q [B,Tq,H,dn+dr], k [B,Tk,Hk,dn], kr [B,Tk,Hr,dr], v [B,Tk,Hk,dv].
struct MlaArgs {
    const void *q, *k, *kr, *v;
    const int *lens; // [B] keys of each sequence, or null (Tk)
    int B, Tq, Tk, H, Hk, Hr, dn, dr, dv;
    int pair; // a workgroup takes a long and a short block instead of one (set at the launch)
    float scale;
};
struct MlaFwdArgs {
    MlaArgs s;
    void *o;
    float *lse; // [B,Tq,H], may be null
};
struct MlaBwdArgs {
    MlaArgs s;
    const void *o, *dout;
    const float *lse;
    float *delta; // workspace [B,H,Tq]: sum of do * o
    void *dq, *dk, *dv, *dkr;
    float *dkr_part; // workspace [B,Tk,Hk,dr] when Hr < Hk, else null
};

// Absorbed heads over the paged cache: q [N,S,H,dl+dr], cache [pages,page,dl+dr].
struct MlaStepArgs {
    const void *q, *cache;
    const int *table, *lens;
    void *o;
    float *lse; // may be null
    int N, S, H, dl, dr, pages, page, cols;
    float scale;
    int mt, units;  // blocks of 16 rows per workgroup; shares the cached rows are cut into
    int tile;       // log2 of a tile's rows; a share is a whole number of tiles
    float *part;    // workspace [2 * units][S * H][dl]
    float *part_ml; // workspace [2 * units][S * H][2]
};

struct NormRopeArgs {
    const void *x, *dy;
    const float *w;
    const int *pos;
    const double *freqs;
    void *y; // y (forward) or dx (backward)
    float *dw, *dw_part;
    long long M; // tokens
    int H, d, r, norm, inter;
    float eps;
    int nblk; // workgroups of the backward (rows of dw_part)
};

struct MlaWriteArgs {
    const void *c, *kr;
    const float *w;
    const int *pos, *slots;
    const double *freqs;
    void *cache;
    long long n_slots;
    int n, dl, dr, norm, inter;
    float eps;
};

struct PagePlanArgs {
    const int *lens, *fresh;
    int *table, *stack;
    const int *n_free;
    int *lens_out, *n_free_out, *granted, *starts, *slots, *positions;
    int N, cols, F, page, cap;
};

// Elements between the rows of an LDS tile beside its columns. bf16: row strides
// of an odd number of 32-byte groups, so that the 32-byte pieces of eight rows
// that a transposing read touches lie in all 64 banks (B2 H16 T2048, forward and
// backward: 227 us with 8 elements, 210 with 16; T16384, 128 + 64 | 128: 6.56
// and 6.46 ms).
template <bool BF> constexpr int MLA_PAD = BF ? 16 : 4;

// How the attention launches share out their blocks (MI355X: 256 CUs).
// A causal walk is as long as its block is late, so two blocks of opposite
// length make one workgroup (MlaArgs::pair) once that still leaves one for
// every CU: equal workgroups, no tail (B8 H16 T4096, 56 + 32 | 56: 2.07 ms
// forward and backward unpaired, 1.94 paired; B2 T512: 60 us unpaired, 66
// paired). Large blocks (32 rows a wave; eight waves for wide heads) reuse
// each LDS read twice, small ones (16 rows, four waves) make two to four times
// as many workgroups: large when, paired, they fill every CU with as many
// workgroups as it holds (per_cu) (B2 T4096 128 + 64 | 128: 1.04 against
// 1.28 ms; B1 T2048: 0.43 against 0.27).
constexpr long long MLA_CUS = 256;
inline long long mla_blocks(long long n, int rows) { return (n + rows - 1) / rows; }
inline bool mla_large(long long heads, long long n, int rows, int per_cu) {
    return heads * mla_blocks(n, rows) >= 2 * MLA_CUS * per_cu;
}
// Waves of a large block: eight share a tile where its registers in flight
// would not fit beside the operands of four (192 | 128: forward 1.59 ms with
// four, 1.46 with eight; query gradients 2.74 and 2.28 ms, T 16384).
constexpr int mla_waves(int dp, int dvp) { return dp + dvp > 224 ? 8 : 4; }
// Where blocks of four times 16 rows leave the chip half empty, the waves of a
// workgroup share rows instead and split every tile of the walk, joining their
// sums at the end: two waves to 16 rows up to two such workgroups per CU (B1
// T512, 16 heads 56 + 32 | 56, forward and backward: 52 us without, 44 with;
// 1024 blocks: 55 and 69 us forward), four, and tiles of 128, where each then
// has a CU to itself, or half of one and much to do: fp32 products, or a long
// walk (B1 T1024, 16 heads on 4, key gradients: 97 us without, 66 with two, 50
// with four; T2048: 186, 126, 104; T512, 16 heads: 19, 16, 20).
constexpr int mla_tile(int split) { return split == 4 ? 128 : 64; }
template <bool BF> constexpr bool mla_fits4(int dp, int dvp) { // (the tiles in LDS)
    return mla_tile(4) * (dp + dvp + 2 * MLA_PAD<BF>) * (int)sizeof(typename Op<BF>::S) <= 96 * 1024;
}
template <bool BF> int mla_split(long long heads, long long n, long long walk, int dp, int dvp) {
    const long long w = heads * mla_blocks(n, 16);
    if (mla_fits4<BF>(dp, dvp) && (w <= MLA_CUS || (w <= 2 * MLA_CUS && (!BF || walk >= 2048)))) return 4;
    return heads * mla_blocks(n, 64) <= 2 * MLA_CUS ? 2 : 1;
}
// Workgroups of a launch over blocks of `rows`; sets pair.
inline long long mla_work(MlaArgs &s, long long heads, long long n, int rows) {
    const long long blocks = mla_blocks(n, rows);
    s.pair = heads * blocks >= 2 * MLA_CUS;
    return heads * (s.pair ? (blocks + 1) / 2 : blocks);
}

// Padded widths the attention kernels are built for: queries and keys, values.
struct MlaPad {
    int d, dv;
};
MlaPad mla_pad(const MlaArgs &s);
void mla_step_plan(MlaStepArgs &a, bool bf16, int cus); // sets mt and units from the sizes
long long mla_step_groups(const MlaStepArgs &a);        // workgroups of the step's larger launch

// workgroups of the backward of norm_rope: one row of dw partial sums each
int norm_rope_blocks(long long rows, int d);

hipError_t launch_mla_fwd_bf16(const MlaFwdArgs &a, hipStream_t st);
hipError_t launch_mla_fwd_f32(const MlaFwdArgs &a, hipStream_t st);
hipError_t launch_mla_bwd_q_bf16(const MlaBwdArgs &a, hipStream_t st);
hipError_t launch_mla_bwd_q_f32(const MlaBwdArgs &a, hipStream_t st);
hipError_t launch_mla_bwd_k_bf16(const MlaBwdArgs &a, hipStream_t st);
hipError_t launch_mla_bwd_k_f32(const MlaBwdArgs &a, hipStream_t st);
hipError_t launch_mla_rope_sum(const MlaBwdArgs &a, bool bf16, hipStream_t st);
hipError_t launch_mla_step(const MlaStepArgs &a, bool bf16, hipStream_t st);
hipError_t launch_mla_join(const MlaStepArgs &a, bool bf16, hipStream_t st);
hipError_t launch_norm_rope(const NormRopeArgs &a, bool bf16, hipStream_t st);
hipError_t launch_norm_rope_bwd(const NormRopeArgs &a, bool bf16, hipStream_t st);
hipError_t launch_norm_sum(const NormRopeArgs &a, hipStream_t st);
hipError_t launch_mla_write(const MlaWriteArgs &a, bool bf16, hipStream_t st);
hipError_t launch_page_plan(const PagePlanArgs &a, hipStream_t st);
hipError_t launch_page_fill(const PagePlanArgs &a, hipStream_t st);
bool page_fill_separate(int cap); // the slots are filled by a launch of their own

// ---------------------------------------------------------------- device code

// Eight consecutive K values of one row (or column) of a 16-wide MFMA
// operand: lane 16g + r holds row r, K = 8g .. 8g + 7. One bf16 MFMA takes
// all 32 K values at once; in fp32 eight 16x16x4 MFMAs take value j of every
// lane in turn (K = {j, 8 + j, 16 + j, 24 + j}), which sums the same products
// as long as both operands are held this way.
template <bool BF> struct Frag;
template <> struct Frag<true> {
    bf16x8 v;
};
template <> struct Frag<false> {
    f32x4 lo, hi;
};
__device__ __forceinline__ f32x4 mma8(const Frag<true> &a, const Frag<true> &b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma8(const Frag<false> &a, const Frag<false> &b, f32x4 c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.lo[j], b.lo[j], c, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.hi[j], b.hi[j], c, 0, 0, 0);
    return c;
}
// eight values stored one after the other (LDS or global, 16-byte aligned)
__device__ __forceinline__ Frag<true> row8(const u16 *p) { return {*reinterpret_cast<const bf16x8 *>(p)}; }
__device__ __forceinline__ Frag<false> row8(const float *p) {
    return {*reinterpret_cast<const f32x4 *>(p), *reinterpret_cast<const f32x4 *>(p + 4)};
}
// Sixteen bytes in registers, and their load from global memory (said so
// explicitly: a pointer picked from several would be read by flat loads, which
// also hold up LDS waits).
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x4 load16(const void *p) {
    return *(const __attribute__((address_space(1))) u32x4 *)p;
}
// sixteen bytes of zeros: where padding columns and absent rows are loaded from
__device__ const u32x4 mla_zeros = {0u, 0u, 0u, 0u};

// row8 from global memory, zeros unless `in`: chosen by address, since a load
// behind a branch is waited for before the next is requested.
__device__ __forceinline__ Frag<true> row8_if(bool in, const u16 *p) {
    return {__builtin_bit_cast(bf16x8, load16(in ? (const void *)p : (const void *)&mla_zeros))};
}
__device__ __forceinline__ Frag<false> row8_if(bool in, const float *p) {
    return {__builtin_bit_cast(f32x4, load16(in ? (const void *)p : (const void *)&mla_zeros)),
            __builtin_bit_cast(f32x4, load16(in ? (const void *)(p + 4) : (const void *)&mla_zeros))};
}

// sum of the eight products, in fp32
__device__ __forceinline__ float dot8(const Frag<true> &a, const Frag<true> &b) {
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) x = fmaf((float)a.v[e], (float)b.v[e], x);
    return x;
}
__device__ __forceinline__ float dot8(const Frag<false> &a, const Frag<false> &b) {
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) x = fmaf(a.lo[e], b.lo[e], x);
#pragma unroll
    for (int e = 0; e < 4; ++e) x = fmaf(a.hi[e], b.hi[e], x);
    return x;
}

// Operand column m0 + lane % 16 of an LDS matrix X[k][m] over the 32 rows from
// k0, in the K order of two accumulator tiles (acc8): lane group g takes rows
// k0 + 4g + e, then k0 + 16 + 4g + e.
__device__ __forceinline__ Frag<true> col8(const u16 *X, int ld, int k0, int m0, int lane) {
    return {join8(operand_tr4(X, ld, k0, m0, lane), operand_tr4(X, ld, k0 + 16, m0, lane))};
}
__device__ __forceinline__ Frag<false> col8(const float *X, int ld, int k0, int m0, int lane) {
    const float *p = X + (k0 + 4 * (lane >> 4)) * ld + m0 + (lane & 15);
    Frag<false> f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f.lo[e] = p[e * ld];
        f.hi[e] = p[(16 + e) * ld];
    }
    return f;
}
// Two 16x16 accumulator tiles (rows k0 .. and k0 + 16 .. of one column block)
// as the other operand of such a product. In bf16 the values are rounded to
// nearest even here: it is what lets the product run on bf16 MFMAs.
template <bool BF> __device__ __forceinline__ Frag<BF> acc8(f32x4 t0, f32x4 t1);
template <> __device__ __forceinline__ Frag<true> acc8<true>(f32x4 t0, f32x4 t1) {
    return {join8(pack4(t0), pack4(t1))};
}
template <> __device__ __forceinline__ Frag<false> acc8<false>(f32x4 t0, f32x4 t1) { return {t0, t1}; }

// x of the three lanes 16, 32 and 48 away folded in: every lane of a column
// (lane % 16) gets the maximum (sum) over its four lane groups.
__device__ __forceinline__ float max4g(float x) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum4g(float x) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// Four consecutive output values.
__device__ __forceinline__ void store4(u16 *p, f32x4 x) {
    uint2 w;
    w.x = f2bf2(x[0], x[1]);
    w.y = f2bf2(x[2], x[3]);
    *reinterpret_cast<uint2 *>(p) = w;
}
__device__ __forceinline__ void store4(float *p, f32x4 x) { *reinterpret_cast<f32x4 *>(p) = x; }

// Workgroup barrier that waits for this wave's LDS accesses only: global
// loads already in flight into registers stay in flight.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Adds the accumulators of the WS waves that share rows, through LDS (64 * T * N
// f32x4 for every group of waves: the tile's own size); true for the one that
// has the sums.
template <int N, int T, int WS>
__device__ __forceinline__ bool join_parts(f32x4 (&x)[T][N], f32x4 *X, int wg, int wu, int lane) {
    f32x4 *p = X + wg * T * N * 64 + lane;
#pragma unroll 1
    for (int w = 1; w < WS; ++w) {
        lds_barrier(); // the last tile's, or part's, readers are done
        if (wu == w) {
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int v = 0; v < N; ++v) p[(t * N + v) * 64] = x[t][v];
        }
        lds_barrier();
        if (wu == 0) {
#pragma unroll
            for (int t = 0; t < T; ++t)
#pragma unroll
                for (int v = 0; v < N; ++v) x[t][v] += p[(t * N + v) * 64];
        }
    }
    return wu == 0;
}

// Keeps the compiler from moving instructions across: what is requested before
// it is in flight during what comes after. Without it the compiler, short of
// registers, sinks every LDS read to just before its use and waits for it.
__device__ __forceinline__ void in_flight() { __builtin_amdgcn_sched_barrier(0); }

// N operands along K of the 16 rows at p (row stride ld), for this lane.
template <bool BF, int N> struct Frags {
    Frag<BF> f[N];
    __device__ __forceinline__ void rows(const typename Op<BF>::S *X, int ld, int row0, int lane) {
        const typename Op<BF>::S *p = X + (row0 + (lane & 15)) * ld + 8 * (lane >> 4);
#pragma unroll
        for (int k = 0; k < N; ++k) f[k] = row8(p + 32 * k);
    }
    // N operand columns of 16 from column m0 on, over the 32 rows from k0
    __device__ __forceinline__ void cols(const typename Op<BF>::S *X, int ld, int k0, int m0, int lane) {
#pragma unroll
        for (int v = 0; v < N; ++v) f[v] = col8(X, ld, k0, m0 + 16 * v, lane);
    }
};

// Rows of a sequence, NR at a time, from global memory over registers into an
// LDS tile [NR][ld]: columns 0 .. d0 - 1 from x0, d0 .. d0 + d1 - 1 from x1
// (both multiples of 8), zeros up to DP and for rows past the end. A thread
// has one 16-byte column of every RP-th row, so its source and row stride are
// fixed (padding columns: the zeros above, with stride 0). fetch() only issues
// the loads (rows past the end read the last one), without a branch that would
// have them waited for; stash() masks and writes.
template <bool BF, int DP, int NR, int NT> struct RowTile {
    using S = typename Op<BF>::S;
    static constexpr int V = Op<BF>::VEC;
    static constexpr int NG = DP / V;
    static constexpr int RP = NT / NG, NIT = (NR + RP - 1) / RP;
    u32x4 r[NIT];
    const S *p;
    unsigned rs;
    int j0, c;
    __device__ __forceinline__ void init(const S *x0, size_t rs0, int d0, const S *x1, size_t rs1, int d1, int tid) {
        c = (tid % NG) * V;
        j0 = tid < RP * NG ? tid / NG : NR; // (the threads left over write nothing)
        p = c < d0 ? x0 + c : c < d0 + d1 ? x1 + (c - d0) : (const S *)&mla_zeros;
        rs = c < d0 ? (unsigned)rs0 : c < d0 + d1 ? (unsigned)rs1 : 0u;
    }
    // from row row0 on, of n rows (n >= 1), `shift` elements further (another head)
    __device__ __forceinline__ void fetch(int row0, int n, size_t shift = 0) {
        const S *q = p + (rs ? shift : 0);
#pragma unroll
        for (int m = 0; m < NIT; ++m)
            r[m] = load16(q + (size_t)(unsigned)min(row0 + j0 + m * RP, n - 1) * rs);
    }
    __device__ __forceinline__ void stash(S *dst, int ld, int row0, int n) {
        S *q = dst + j0 * ld + c;
        if (row0 + NR > n) { // (the last tile)
#pragma unroll
            for (int m = 0; m < NIT; ++m)
                if (row0 + j0 + m * RP >= n) r[m] = u32x4{0u, 0u, 0u, 0u};
        }
#pragma unroll
        for (int m = 0; m < NIT; ++m)
            if (j0 + m * RP < NR) *reinterpret_cast<u32x4 *>(q + m * RP * ld) = r[m];
    }
};

// Workgroup -> (batch-head, block of its sequence), longest walks first.
// Workgroups go round robin over the 8 XCDs: eight heads at a time run side by
// side, one per XCD, so that a head's rows are read into one L2; what is left
// over (fewer than eight heads) is dealt out block by block, which keeps the
// XCDs equally loaded when there are few heads (four heads of 128 causal
// blocks, two XCDs each: half a head per XCD would give one of the two three
// times the work of the other).
__device__ __forceinline__ void head_block(int id, int heads, int blocks, int &bh, int &blk) {
    const int full = heads / 8 * 8;
    if (id < full * blocks) {
        bh = id / (8 * blocks) * 8 + id % 8;
        blk = id / 8 % blocks;
    } else {
        const int i = id - full * blocks;
        bh = full + i % (heads - full);
        blk = i / (heads - full);
    }
}

} // namespace gdn
