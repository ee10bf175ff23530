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
long long mla_weights_groups(const MlaWeightsArgs &a);
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
    // segment: kept rows before it, rows of the threshold's weight before it, done
    int *ticket, *kept, *ties, *done;
    uint32_t *bar; // key of the lightest row kept
    int *spare;    // how many rows of that key are kept
    int segs;      // segments of a sequence
};
constexpr int EVICT_ROW16 = 144; // widest row
// Rows of a segment: what a workgroup of the move holds in registers.
__host__ __device__ constexpr int evict_segment(int row16) { return row16 <= 72 ? 256 : 128; }
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
    double *sums; // [rows][nch] sums of a piece, relative to its largest logit
    float *tops;  // [rows][nch]
    int *best;    // [rows][nch] first place of the largest
    double *left; // [N][nch] sums of what a rejected draft leaves
    double *pick; // [N][PICK]: what was decided
};
constexpr int VERIFY_PICK = 8;
int verify_pieces(int V, bool bf16); // pieces of a row
hipError_t launch_verify_sums(const VerifyArgs &a, bool bf16, hipStream_t st);
hipError_t launch_verify_left(const VerifyArgs &a, bool bf16, hipStream_t st);
hipError_t launch_verify_draw(const VerifyArgs &a, bool bf16, hipStream_t st);

} // namespace gdn
