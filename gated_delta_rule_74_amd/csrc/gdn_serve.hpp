// Serving beside the plain step: argument blocks and launch interface of the
// kernels for shared prefixes, cached rows' weights, eviction, page return,
// draft verification and the state after accepted tokens.
#pragma once

#include "gdn_mla.hpp"

namespace gdn {

// kinds of launches, as listed at gdn_launch_kind
enum ServeKind {
    K_MLA_PREFIX = 20,
    K_MLA_WEIGHTS,
    K_EVICT_CHOOSE,
    K_EVICT_MOVE,
    K_PAGE_TRIM,
    K_VERIFY_SUMS,
    K_VERIFY_DECIDE,
    K_VERIFY_LEFT,
    K_VERIFY_DRAW,
    K_STEP_COMMIT
};

// Queries of a batch against prefixes that groups of its sequences share.
struct PrefixArgs {
    const void *q, *cache;
    const int *table, *plens, *starts; // [G,cols], [G], [G+1]
    int N, S, H, dl, dr, pages, page, cols, G;
    float scale;
    int qt, qb;    // blocks of 16 queries a wave; queries of a workgroup
    int units;     // workgroups: shares the blocks' walks are cut into
    float *part;   // workspace [units + blocks][qb][dl]
    float *part_ml; // workspace [units + blocks][qb][2]
    // 1: the sequences' own rows are walked here too, after the groups; else by mla_step_kernel
    int own;
    const int *own_table, *lens; // [N,own_cols], [N]
    int own_cols, own_blocks, own_qb; // blocks of a sequence's queries, queries of its parts
    float *own_part;   // workspace [units + N own_blocks][own_qb][dl]
    float *own_part_ml; // workspace [units + N own_blocks][own_qb][2]
    long long *walks;  // workspace [N][2]: where a sequence's walk begins, the share (of sequences with rows)
};
void mla_prefix_plan(PrefixArgs &a, bool bf16, int cus); // sets qt, qb and units
long long mla_prefix_blocks(const PrefixArgs &a);        // blocks of queries there may be
hipError_t launch_mla_prefix_bf16(const PrefixArgs &a, hipStream_t st);
hipError_t launch_mla_prefix_f32(const PrefixArgs &a, hipStream_t st);
long long mla_shared_join_groups(const MlaStepArgs &a);
hipError_t launch_mla_shared_join(const MlaStepArgs &a, const PrefixArgs &p, bool bf16, hipStream_t st);

// h [N,H,dk,dv] after the first counts[n] of S tokens.
struct CommitArgs {
    const void *k, *v;
    const float *g, *beta, *A_log, *h_in;
    const int *counts;
    float *h_out;
    int N, S, H, dk, dv, additive, logits, l2k;
};
long long step_commit_groups(int N, int H, int dv); // workgroups of 256 threads
hipError_t launch_step_commit(const CommitArgs &a, bool bf16, hipStream_t st);

struct PageTrimArgs {
    const int *lens, *fresh, *table;
    int *stack;
    const int *n_free;
    int *n_free_out;
    int N, cols, F, page;
};
hipError_t launch_page_trim(const PageTrimArgs &a, hipStream_t st);

// Weights of cached rows: q [N,S,H,dl+dr] against the paged cache.
struct MlaWeightsArgs {
    const void *q, *cache;
    const int *table, *lens, *known; // known may be null (lens - S)
    const float *lse;
    float *weights;
    int N, S, H, d, pages, page, cols;
    float scale, decay;
};
long long mla_weights_groups(const MlaWeightsArgs &a, bool bf16);
hipError_t launch_mla_weights(const MlaWeightsArgs &a, bool bf16, hipStream_t st);

// Rows that an eviction keeps, and their move to the front.
struct EvictArgs {
    const int *table, *lens, *keep;
    float *weights;
    void *cache;
    int *lens_out;
    int N, cols, pages, page, row16; // row16: 16-byte pieces of a cache row
    int first, recent;
    // workspace, per sequence: ticket counter, threshold; per sequence and
    // grain: kept rows before it, rows of the threshold's weight before it; per sequence and segment: done
    int *ticket, *kept, *ties, *done;
    uint32_t *bar; // key of the lightest row kept
    int *spare;    // how many rows of that key are kept
    int segs, grains; // segments and grains of a sequence
    // where several workgroups choose for a sequence (chunks > 1): their histograms, two passes' of them, what the
    // digits found so far leave, and how many are done
    int chunks;
    int *hist;       // [2][N][chunks][EVICT_BINS]
    uint32_t *state; // [N][3][2]: digits found, rows wanted among those that agree
    int *arrived;    // [N]
};
constexpr int EVICT_ROW16 = 144; // widest row
// Rows of a segment: what a workgroup of the move holds in registers.
constexpr int EVICT_MOVE = 256;    // threads of the move
constexpr int EVICT_HELD = 18;     // 16-byte pieces that each of them holds
__host__ __device__ constexpr int evict_segment(int row16) {
    const int most = EVICT_MOVE * EVICT_HELD / row16;
    return most >= 256 ? 256 : most >= 128 ? 128 : most >= 64 ? 64 : 32;
}
// Rows that are counted together: a segment's, or a part of them.
__host__ __device__ constexpr int evict_grain(int row16) { return evict_segment(row16) < 64 ? evict_segment(row16) : 64; }
constexpr int EVICT_CHUNK = 8192;  // rows of a workgroup of the choice, where several take a sequence
constexpr long long EVICT_ONE = 32768; // longest sequence that one takes
constexpr int EVICT_BINS = 2048;   // values of a digit
inline int evict_chunks(long long rows) { return rows <= EVICT_ONE ? 1 : (int)((rows + EVICT_CHUNK - 1) / EVICT_CHUNK); }
hipError_t launch_evict_choose(const EvictArgs &a, hipStream_t st);
hipError_t launch_evict_move(const EvictArgs &a, hipStream_t st);

struct VerifyArgs {
    const void *logits, *dlogits; // dlogits may be null
    const int *draft, *dlens;     // dlens may be null
    const float *temp, *uniforms; // temp may be null
    int *accepted, *tokens;
    float *logprobs; // may be null
    int N, S, V, nch;
    // workspace: rows [N * (S + 1)] of the target, then [N * S] of the draft
    double *sums; // [rows][nch] sums of a piece's exponentials, relative to
    float *refs;  // [rows][nch] this logit
    float *tops;  // [rows][nch] its largest logit
    int *best;    // [rows][nch] first place of the largest
    double *left; // [N][nch] sums of what a rejected draft leaves
    double *pick; // [N][PICK]: what was decided
};
constexpr int VERIFY_PICK = 8;
int verify_pieces(int V); // pieces of a row
hipError_t launch_verify_sums(const VerifyArgs &a, bool bf16, hipStream_t st);
hipError_t launch_verify_decide(const VerifyArgs &a, bool bf16, hipStream_t st);
hipError_t launch_verify_left(const VerifyArgs &a, bool bf16, hipStream_t st);
hipError_t launch_verify_draw(const VerifyArgs &a, bool bf16, hipStream_t st);

// ---------------------------------------------------------------- device code

// Sequences of parts(n) >= 0 equal pieces each, end to end: which sequence
// holds piece b (n), and which of its pieces that is; false: there is no such piece. So the
// workgroups with work are the first ones, which spread over the XCDs whatever the
// lengths are (with a grid of sequences times their longest, every eighth
// workgroup an XCD: 12 sequences of up to 2000 rows, 32 queries of fp32, 57 us; so 33). Every wave finds out for itself.
struct Pieces {
    int N, per, before, mine; // sequences a lane adds up; pieces before its own, and of its own
    int total;
    template <class F> __device__ __forceinline__ static Pieces of(int N, F &&parts, int lane) {
        Pieces s = {N, (N + 63) / 64, 0, 0, 0};
        const int from = min(lane * s.per, N), to = min(from + s.per, N);
#pragma unroll 4
        for (int i = from; i < to; ++i) s.mine += parts(i);
        s.sum(lane);
        return s;
    }
    __device__ __forceinline__ void sum(int lane) {
        int x = mine;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int y = __shfl_up(x, o, 64);
            if (lane >= o) x += y;
        }
        before = x - mine;
        total = __builtin_amdgcn_readlane(x, 63);
    }
    // the sequence of piece b < total, and which of its pieces that is
    template <class F> __device__ __forceinline__ void find(F &&parts, int b, int lane, int &n, int &piece) const {
        int l = __builtin_ctzll(__ballot(before + mine > b)), first = l * per, many = min(per, N - first);
        b -= __builtin_amdgcn_readlane(before, l);
        while (many > 1) { // (a 64th of them at a time)
            Pieces s = of(many, [&](int i) { return parts(first + i); }, lane);
            l = __builtin_ctzll(__ballot(s.before + s.mine > b));
            b -= __builtin_amdgcn_readlane(s.before, l);
            first += l * s.per;
            many = min(s.per, many - l * s.per);
        }
        n = first;
        piece = b;
    }
};
template <class F> __device__ __forceinline__ bool find_piece(int N, F &&parts, int b, int lane, int &n, int &piece) {
    const Pieces s = Pieces::of(N, parts, lane);
    if (b >= s.total) return false;
    s.find(parts, b, lane, n, piece);
    return true;
}

} // namespace gdn
