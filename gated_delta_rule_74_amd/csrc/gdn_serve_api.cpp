// C ABI of the operators beside the plain step that deal with sequences as a
// whole: accepted tokens' states, eviction, page return and draft
// verification. The operations are described in include/gdn.h.
#include "gdn.h"

#include <hip/hip_runtime.h>

#include "gdn_check.hpp"
#include "gdn_serve.hpp"

using namespace gdn::check;

namespace {

constexpr uint32_t STEP_FLAGS = GDN_FLAG_ADDITIVE | GDN_FLAG_GATE_LOGITS | GDN_FLAG_L2NORM_K;

gdn_status_t check_space(const char *func, const void *ws, size_t ws_bytes, size_t need) {
    if (need && (!ws || ws_bytes < need))
        return fail(GDN_EWORKSPACE, "%s needs %zu bytes of workspace, got %zu", func, need, ws ? ws_bytes : 0);
    if (need && (uintptr_t)ws % 256) return fail(GDN_EINVAL, "workspace must be 256-byte aligned");
    return GDN_OK;
}

// A workspace handed out piece by piece; without one, only their sizes are added up.
struct Carve {
    char *p;
    size_t used = 0;
    template <class T> T *take(size_t n) {
        T *at = p ? (T *)(p + used) : nullptr;
        used += align_up(n * sizeof(T));
        return at;
    }
};

gdn_status_t check_evict(int32_t N, int32_t max_pages, int32_t page_size, int32_t row_bytes) {
    if (N < 0 || max_pages < 1 || page_size < 1) return fail(GDN_EINVAL, "N must be >= 0, max_pages and page_size >= 1");
    if (row_bytes < 16 || row_bytes % 16) return fail(GDN_EINVAL, "row_bytes must be a multiple of 16");
    if (row_bytes > 16 * gdn::EVICT_ROW16)
        return fail(GDN_EUNSUPPORTED, "row_bytes must be at most %d", 16 * gdn::EVICT_ROW16);
    // (the end of a sequence's last chunk stays in int32)
    if ((double)max_pages * page_size > LIMIT - gdn::EVICT_CHUNK || (double)N * max_pages >= LIMIT)
        return fail(GDN_EINVAL, "table too large");
    // (segments are counted in int32; one workgroup of 1024 threads for every chunk)
    const double rows = (double)max_pages * page_size;
    if (N * (rows / 32 + 1) >= LIMIT / 2 || N * (rows / gdn::EVICT_CHUNK + 1) * 1024 >= THREADS)
        return fail(GDN_EINVAL, "too many rows for a launch");
    return GDN_OK;
}
size_t carve_evict(gdn::EvictArgs &a, void *ws) {
    const int seg = gdn::evict_segment(a.row16);
    a.segs = (int)(((long long)a.cols * a.page + seg - 1) / seg);
    const int grain = gdn::evict_grain(a.row16);
    a.grains = (int)(((long long)a.cols * a.page + grain - 1) / grain);
    const size_t n = a.N;
    Carve c{(char *)ws};
    a.ticket = c.take<int>(n);
    a.bar = c.take<uint32_t>(n);
    a.spare = c.take<int>(n);
    a.kept = c.take<int>(n * a.grains);
    a.ties = c.take<int>(n * a.grains);
    a.done = c.take<int>(n * a.segs);
    a.chunks = gdn::evict_chunks((long long)a.cols * a.page);
    if (a.chunks > 1) {
        a.hist = c.take<int>(2 * n * a.chunks * gdn::EVICT_BINS);
        a.state = c.take<uint32_t>(n * 3 * 2);
        a.arrived = c.take<int>(n);
    }
    return c.used;
}

gdn_status_t check_verify(int32_t N, int32_t S, int32_t V, int32_t dtype) {
    if (N < 0 || S < 0 || V < 1) return fail(GDN_EINVAL, "N, S must be >= 0 and V >= 1");
    if (dtype != GDN_F32 && dtype != GDN_BF16) return fail(GDN_EINVAL, "unknown dtype %d", dtype);
    if ((double)N * ((double)S + 1) * V >= LIMIT || V > (1 << 26) || S > (1 << 30))
        return fail(GDN_EINVAL, "logits too large");
    if ((double)N * (2.0 * S + 2) * (gdn::verify_pieces(V) + 4.0) * 64 >= THREADS)
        return fail(GDN_EINVAL, "too many rows for a launch");
    return GDN_OK;
}
size_t carve_verify(gdn::VerifyArgs &a, void *ws) {
    const size_t rows = (size_t)a.N * (2 * (size_t)a.S + 1);
    Carve c{(char *)ws};
    a.sums = c.take<double>(rows * a.nch);
    a.left = c.take<double>((size_t)a.N * a.nch);
    a.pick = c.take<double>((size_t)a.N * gdn::VERIFY_PICK);
    a.tops = c.take<float>(rows * a.nch);
    a.refs = c.take<float>(rows * a.nch);
    a.best = c.take<int>(rows * a.nch);
    return c.used;
}

} // namespace

extern "C" {

gdn_status_t gdn_step_commit(int32_t N, int32_t S, int32_t H, int32_t dk, int32_t dv, int32_t dtype, uint32_t flags,
                             const void *k, const void *v, const float *g, const float *beta, const float *A_log,
                             const int32_t *counts, const float *h_in, float *h_out, void *stream) {
    if (N < 0 || H < 1 || S < 0) return fail(GDN_EINVAL, "N, S must be >= 0 and H >= 1");
    if (dk < 1 || dv < 1 || dk > 128 || dv > 128) return fail(GDN_EINVAL, "dk and dv must be in [1, 128]");
    if (dtype != GDN_F32 && dtype != GDN_BF16) return fail(GDN_EINVAL, "unknown dtype %d", dtype);
    if (flags & ~STEP_FLAGS) return fail(GDN_EINVAL, "unknown flag bits 0x%x", flags);
    if ((double)N * H * dk * dv >= LIMIT || (double)N * S * H * (dk > dv ? dk : dv) >= LIMIT)
        return fail(GDN_EINVAL, "state or tokens too large");
    if (S > 0 && (double)gdn::step_commit_groups(N, H, dv) * 256 >= THREADS)
        return fail(GDN_EINVAL, "too many states for a launch");
    const size_t e = esize(dtype), n = (size_t)N * S * H, state = (size_t)N * H * dk * dv * 4;
    const Buf b[] = {{k, n * dk * e, "k", 4, false, true},
                     {v, n * dv * e, "v", 4, false, true},
                     {g, n * 4, "g", 4, false, true},
                     {beta, n * 4, "beta", 4, false, true},
                     {A_log, n ? (size_t)H * 4 : 0, "A_log", 4, false, true},
                     {counts, n ? (size_t)N * 4 : 0, "counts", 4, false, true},
                     {h_in, state, "h_in", 4, false, false},
                     {h_out, state, "h_out", 4, true, true}};
    const int same[1][2] = {{6, 7}}; // in place: a wave reads its part of the state whole before it writes it
    const gdn_status_t st = check_bufs(b, 8, same, 1);
    if (st != GDN_OK) return st;
    if (N == 0) return ok();
    hipStream_t strm = (hipStream_t)stream;
    if (S == 0) { // no token: the states are carried over
        if (h_in == h_out) return ok();
        return hip_status(gdn::launch_copy_or_zero(h_out, h_in, state / 4, strm), "gdn_step_commit (no token)");
    }
    gdn::CommitArgs a;
    a.k = k;
    a.v = v;
    a.g = g;
    a.beta = beta;
    a.A_log = A_log;
    a.counts = counts;
    a.h_in = h_in;
    a.h_out = h_out;
    a.N = N;
    a.S = S;
    a.H = H;
    a.dk = dk;
    a.dv = dv;
    a.additive = (flags & GDN_FLAG_ADDITIVE) ? 1 : 0;
    a.logits = (flags & GDN_FLAG_GATE_LOGITS) ? 1 : 0;
    a.l2k = (flags & GDN_FLAG_L2NORM_K) ? 1 : 0;
    return hip_status(gdn::bracketed(
                          gdn::K_STEP_COMMIT, [&] { return gdn::launch_step_commit(a, dtype == GDN_BF16, strm); }, strm),
                      "gdn_step_commit launch");
}

size_t gdn_mla_evict_workspace_size(int32_t N, int32_t max_pages, int32_t page_size, int32_t row_bytes) {
    if (check_evict(N, max_pages, page_size, row_bytes) != GDN_OK || N == 0) return 0;
    gdn::EvictArgs a = {};
    a.N = N;
    a.cols = max_pages;
    a.page = page_size;
    a.row16 = row_bytes / 16;
    return carve_evict(a, nullptr);
}

gdn_status_t gdn_mla_evict(int32_t N, int32_t max_pages, int32_t pages, int32_t page_size, int32_t row_bytes,
                           int32_t first, int32_t recent, const int32_t *block_table, const int32_t *lens,
                           const int32_t *keep, float *weights, void *cache, int32_t *lens_out, void *ws,
                           size_t ws_bytes, void *stream) {
    gdn_status_t st = check_evict(N, max_pages, page_size, row_bytes);
    if (st != GDN_OK) return st;
    if (pages < 1 || (double)pages * page_size >= LIMIT) return fail(GDN_EINVAL, "pages must be >= 1, the pool below 2^31 rows");
    if (first < 0 || recent < 0) return fail(GDN_EINVAL, "first and recent must be >= 0");
    const size_t slots = (size_t)pages * page_size, need = gdn_mla_evict_workspace_size(N, max_pages, page_size, row_bytes);
    const bool some = N > 0;
    const Buf b[] = {{block_table, (size_t)N * max_pages * 4, "block_table", 4, false, true},
                     {lens, (size_t)N * 4, "lens", 4, false, true},
                     {keep, (size_t)N * 4, "keep", 4, false, true},
                     {weights, slots * 4, "weights", 4, true, some},
                     {cache, slots * row_bytes, "cache", 16, true, some},
                     {lens_out, (size_t)N * 4, "lens_out", 4, true, true},
                     {ws, need, "workspace", 1, true, false}};
    st = check_bufs(b, 7);
    if (st != GDN_OK) return st;
    if (!some) return ok();
    st = check_space("gdn_mla_evict", ws, ws_bytes, need);
    if (st != GDN_OK) return st;
    gdn::EvictArgs a = {};
    a.table = block_table;
    a.lens = lens;
    a.keep = keep;
    a.weights = weights;
    a.cache = cache;
    a.lens_out = lens_out;
    a.N = N;
    a.cols = max_pages;
    a.pages = pages;
    a.page = page_size;
    a.row16 = row_bytes / 16;
    a.first = first;
    a.recent = recent;
    carve_evict(a, ws);
    hipStream_t strm = (hipStream_t)stream;
    hipError_t e = gdn::bracketed(gdn::K_EVICT_CHOOSE, [&] { return gdn::launch_evict_choose(a, strm); }, strm);
    if (e == hipSuccess) e = gdn::bracketed(gdn::K_EVICT_MOVE, [&] { return gdn::launch_evict_move(a, strm); }, strm);
    return hip_status(e, "gdn_mla_evict launch");
}

gdn_status_t gdn_page_trim(int32_t N, int32_t max_pages, int32_t n_pages, int32_t page_size, const int32_t *lens,
                           const int32_t *new_lens, const int32_t *block_table, int32_t *free_pages,
                           const int32_t *n_free, int32_t *n_free_out, void *stream) {
    if (N < 0 || max_pages < 1 || n_pages < 1 || page_size < 1)
        return fail(GDN_EINVAL, "N must be >= 0, max_pages, n_pages and page_size >= 1");
    if ((double)N * max_pages > LIMIT - AHEAD) return fail(GDN_EINVAL, "table too large");
    const size_t n = (size_t)N * 4;
    const Buf b[] = {{lens, n, "lens", 4, false, true},
                     {new_lens, n, "new_lens", 4, false, true},
                     {block_table, n * max_pages, "block_table", 4, false, true},
                     {n_free, 4, "n_free", 4, false, true},
                     {free_pages, (size_t)n_pages * 4, "free_pages", 4, true, true},
                     {n_free_out, 4, "n_free_out", 4, true, true}};
    const int same[1][2] = {{3, 5}};
    const gdn_status_t st = check_bufs(b, 6, same, 1);
    if (st != GDN_OK) return st;
    const gdn::PageTrimArgs a = {lens, new_lens, block_table, free_pages, n_free, n_free_out, N, max_pages, n_pages, page_size};
    hipStream_t strm = (hipStream_t)stream;
    return hip_status(gdn::bracketed(gdn::K_PAGE_TRIM, [&] { return gdn::launch_page_trim(a, strm); }, strm),
                      "gdn_page_trim launch");
}

size_t gdn_draft_verify_workspace_size(int32_t N, int32_t S, int32_t V, int32_t dtype) {
    if (check_verify(N, S, V, dtype) != GDN_OK || N == 0) return 0;
    gdn::VerifyArgs a = {};
    a.N = N;
    a.S = S;
    a.V = V;
    a.nch = gdn::verify_pieces(V);
    return carve_verify(a, nullptr);
}

gdn_status_t gdn_draft_verify(int32_t N, int32_t S, int32_t V, int32_t dtype, const void *logits, const int32_t *draft,
                              const int32_t *draft_lens, const void *draft_logits, const float *temperature,
                              const float *uniforms, int32_t *accepted, int32_t *tokens, float *logprobs, void *ws,
                              size_t ws_bytes, void *stream) {
    gdn_status_t st = check_verify(N, S, V, dtype);
    if (st != GDN_OK) return st;
    const size_t e = esize(dtype), n = (size_t)N, rows = n * ((size_t)S + 1), drafts = n * S;
    const size_t need = gdn_draft_verify_workspace_size(N, S, V, dtype);
    const Buf b[] = {{logits, rows * V * e, "logits", 4, false, true},
                     {draft, drafts * 4, "draft", 4, false, true},
                     {draft_lens, n * 4, "draft_lens", 4, false, false},
                     {draft_logits, drafts * V * e, "draft_logits", 4, false, false},
                     {temperature, n * 4, "temperature", 4, false, false},
                     {uniforms, rows * 4, "uniforms", 4, false, true},
                     {accepted, n * 4, "accepted", 4, true, true},
                     {tokens, rows * 4, "tokens", 4, true, true},
                     {logprobs, rows * 4, "logprobs", 4, true, false},
                     {ws, need, "workspace", 1, true, false}};
    st = check_bufs(b, 10);
    if (st != GDN_OK) return st;
    if (N == 0) return ok();
    st = check_space("gdn_draft_verify", ws, ws_bytes, need);
    if (st != GDN_OK) return st;
    gdn::VerifyArgs a;
    a.logits = logits;
    a.dlogits = S > 0 ? draft_logits : nullptr;
    a.draft = draft;
    a.dlens = draft_lens;
    a.temp = temperature;
    a.uniforms = uniforms;
    a.accepted = accepted;
    a.tokens = tokens;
    a.logprobs = logprobs;
    a.N = N;
    a.S = S;
    a.V = V;
    a.nch = gdn::verify_pieces(V);
    carve_verify(a, ws);
    const bool bf = dtype == GDN_BF16;
    hipStream_t strm = (hipStream_t)stream;
    hipError_t he = gdn::bracketed(gdn::K_VERIFY_SUMS, [&] { return gdn::launch_verify_sums(a, bf, strm); }, strm);
    if (he == hipSuccess)
        he = gdn::bracketed(gdn::K_VERIFY_DECIDE, [&] { return gdn::launch_verify_decide(a, bf, strm); }, strm);
    if (he == hipSuccess && S > 0) // (without drafts none is rejected)
        he = gdn::bracketed(gdn::K_VERIFY_LEFT, [&] { return gdn::launch_verify_left(a, bf, strm); }, strm);
    if (he == hipSuccess)
        he = gdn::bracketed(gdn::K_VERIFY_DRAW, [&] { return gdn::launch_verify_draw(a, bf, strm); }, strm);
    return hip_status(he, "gdn_draft_verify launch");
}

} // extern "C"
