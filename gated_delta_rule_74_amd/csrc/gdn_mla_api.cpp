// C ABI of the latent-attention and paged-cache operators: argument
// validation, workspace layout and kernel launches. The operations are
// described in include/gdn.h.
#include "gdn.h"

#include <hip/hip_runtime.h>

#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "gdn_mla.hpp"

namespace {

gdn_status_t fail(gdn_status_t st, const char *fmt, ...) {
    char text[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(text, sizeof text, fmt, ap);
    va_end(ap);
    return gdn::fail_detail(st, text);
}
gdn_status_t ok() { return gdn::fail_detail(GDN_OK, ""); }
gdn_status_t hip_status(hipError_t e, const char *what) {
    return e == hipSuccess ? ok() : fail(GDN_EHIP, "%s: %s", what, hipGetErrorString(e));
}

size_t align_up(size_t x) { return (x + 255) & ~(size_t)255; }
size_t esize(int dtype) { return dtype == GDN_BF16 ? 2 : 4; }
constexpr double LIMIT = 2147483648.0; // elements of a tensor
constexpr double THREADS = 4294967296.0; // threads of a launch
// What the kernels add to a position or a count (a few tiles ahead, a thread's
// run) must not pass int32: sizes that bound those stay so much below it.
constexpr double AHEAD = 2048.0;
constexpr int CUS = 256;               // compute units of the chip the kernels are built for

// One buffer of a call.
struct Buf {
    const void *p;
    size_t n;
    const char *name;
    size_t align;
    bool out, need;
};

// Required pointers, alignment, and no output over another buffer. `same`:
// index pair of an input and an output that may be one buffer (-1: none).
gdn_status_t check_bufs(const Buf *b, int n, const int (*same)[2] = nullptr, int nsame = 0) {
    for (int i = 0; i < n; ++i) {
        if (b[i].need && b[i].n && !b[i].p) return fail(GDN_EINVAL, "%s is NULL", b[i].name);
        if (b[i].p && (uintptr_t)b[i].p % b[i].align)
            return fail(GDN_EINVAL, "%s must be %zu-byte aligned", b[i].name, b[i].align);
    }
    for (int i = 0; i < n; ++i)
        for (int j = 0; j < n; ++j) {
            if (!b[i].out || i == j || (b[j].out && j > i)) continue;
            if (!b[i].p || !b[j].p || !b[i].n || !b[j].n) continue;
            bool may = false;
            for (int k = 0; k < nsame; ++k)
                may |= same[k][0] == j && same[k][1] == i && b[i].p == b[j].p;
            const char *x = (const char *)b[i].p, *y = (const char *)b[j].p;
            if (!may && x < y + b[j].n && y < x + b[i].n)
                return fail(GDN_EINVAL, "output %s overlaps %s", b[i].name, b[j].name);
        }
    return GDN_OK;
}

gdn_status_t check_mla(const gdn_mla_shape_t *s) {
    if (!s) return fail(GDN_EINVAL, "shape is NULL");
    if (s->B < 1 || s->H < 1 || s->Hk < 1) return fail(GDN_EINVAL, "B, H and Hk must be >= 1");
    if (s->Tq < 0 || s->Tk < s->Tq) return fail(GDN_EINVAL, "Tk >= Tq >= 0 is required");
    if (s->dtype != GDN_F32 && s->dtype != GDN_BF16) return fail(GDN_EINVAL, "unknown dtype %d", s->dtype);
    if (s->H % s->Hk) return fail(GDN_EINVAL, "Hk must divide H");
    if (s->dr < 0 || (s->dr > 0 && (s->Hr < 1 || s->Hk % s->Hr)))
        return fail(GDN_EINVAL, "Hr must divide Hk (with dr > 0)");
    if (s->dn < 1 || s->dv < 1) return fail(GDN_EINVAL, "dn and dv must be >= 1");
    if (s->dn % 8 || s->dr % 8 || s->dv % 8 || s->dn > 128 || s->dr > 64 || s->dv > 128)
        return fail(GDN_EUNSUPPORTED, "dn, dv must be multiples of 8 up to 128, dr one up to 64");
    if (!(s->scale > 0.f) || !isfinite(s->scale)) return fail(GDN_EINVAL, "scale must be positive and finite");
    // the elements of q, o, k, k_rope and v, each by itself (H may be many times Hk, Tk many times Tq)
    const double qrows = (double)s->B * s->Tq * s->H, krows = (double)s->B * s->Tk * s->Hk;
    const double rrows = s->dr > 0 ? (double)s->B * s->Tk * s->Hr : 0.0;
    if (qrows * (s->dn + s->dr) >= LIMIT || qrows * s->dv >= LIMIT || krows * s->dn >= LIMIT ||
        rrows * s->dr >= LIMIT || krows * s->dv >= LIMIT)
        return fail(GDN_EINVAL, "tensor too large");
    // threads of a launch: a workgroup for every head and 64 rows where there are many
    gdn::MlaArgs a = {};
    a.dn = s->dn;
    a.dr = s->dr;
    a.dv = s->dv;
    const gdn::MlaPad pad = gdn::mla_pad(a);
    const int wide = s->dtype == GDN_BF16 ? 64 * gdn::mla_waves(pad.d, pad.dv) : 256;
    if ((double)s->B * s->H * ((s->Tq + 63) / 64) * wide >= THREADS ||
        (double)s->B * s->Hk * ((s->Tk + 63) / 64) * 256 >= THREADS)
        return fail(GDN_EINVAL, "too many heads for a launch");
    return GDN_OK;
}

gdn::MlaArgs mla_args(const gdn_mla_shape_t *s, const void *q, const void *k, const void *kr, const void *v,
                      const int32_t *lens) {
    gdn::MlaArgs a;
    a.q = q;
    a.k = k;
    a.kr = s->dr > 0 ? kr : nullptr;
    a.v = v;
    a.lens = lens;
    a.B = s->B;
    a.Tq = s->Tq;
    a.Tk = s->Tk;
    a.H = s->H;
    a.Hk = s->Hk;
    a.Hr = s->dr > 0 ? s->Hr : 0;
    a.dn = s->dn;
    a.dr = s->dr;
    a.dv = s->dv;
    a.pair = 0;
    a.scale = s->scale;
    return a;
}

// byte sizes of the tensors of a shape
struct MlaSizes {
    size_t q, k, kr, v, o, lse, lens;
};
MlaSizes mla_sizes(const gdn_mla_shape_t *s) {
    const size_t e = esize(s->dtype), B = s->B, Tq = s->Tq, Tk = s->Tk;
    MlaSizes z;
    z.q = B * Tq * s->H * (s->dn + s->dr) * e;
    z.k = B * Tk * s->Hk * s->dn * e;
    z.kr = s->dr > 0 ? B * Tk * s->Hr * s->dr * e : 0;
    z.v = B * Tk * s->Hk * s->dv * e;
    z.o = B * Tq * s->H * s->dv * e;
    z.lse = B * Tq * s->H * 4;
    z.lens = B * 4;
    return z;
}
size_t mla_delta_bytes(const gdn_mla_shape_t *s) { return align_up((size_t)s->B * s->H * s->Tq * 4); }
size_t mla_part_bytes(const gdn_mla_shape_t *s) {
    return s->dr > 0 && s->Hr < s->Hk ? align_up((size_t)s->B * s->Tk * s->Hk * s->dr * 4) : 0;
}

gdn::MlaStepArgs step_args(const gdn_mla_step_shape_t *s) {
    gdn::MlaStepArgs a = {};
    a.N = s->N;
    a.S = s->S;
    a.H = s->H;
    a.dl = s->dl;
    a.dr = s->dr;
    a.pages = s->pages;
    a.page = s->page_size;
    a.cols = s->max_pages;
    a.scale = s->scale;
    if (s->N > 0 && s->S > 0) gdn::mla_step_plan(a, s->dtype == GDN_BF16, CUS);
    else a.mt = a.units = 0;
    return a;
}

gdn_status_t check_step(const gdn_mla_step_shape_t *s) {
    if (!s) return fail(GDN_EINVAL, "shape is NULL");
    if (s->N < 0 || s->S < 0 || s->H < 1) return fail(GDN_EINVAL, "N, S must be >= 0 and H >= 1");
    if (s->dtype != GDN_F32 && s->dtype != GDN_BF16) return fail(GDN_EINVAL, "unknown dtype %d", s->dtype);
    if (s->dl < 1 || s->dr < 0) return fail(GDN_EINVAL, "dl must be >= 1, dr >= 0");
    if (s->dl % 16 || s->dl > 512 || s->dr % 8 || s->dr > 64)
        return fail(GDN_EUNSUPPORTED, "dl must be a multiple of 16 up to 512, dr one of 8 up to 64");
    if (s->pages < 1 || s->page_size < 1 || s->max_pages < 1)
        return fail(GDN_EINVAL, "pages, page_size and max_pages must be >= 1");
    if ((double)s->pages * s->page_size >= LIMIT || (double)s->max_pages * s->page_size > LIMIT - AHEAD ||
        (double)s->N * s->max_pages >= LIMIT)
        return fail(GDN_EINVAL, "cache or table too large");
    if ((double)s->N * s->S * s->H * (s->dl + s->dr) >= LIMIT ||
        (double)s->N * s->max_pages * s->page_size / 32 + s->N >= LIMIT / 2)
        return fail(GDN_EINVAL, "tokens too large");
    if (!(s->scale > 0.f) || !isfinite(s->scale)) return fail(GDN_EINVAL, "scale must be positive and finite");
    if ((double)gdn::mla_step_groups(step_args(s)) * 256 >= THREADS)
        return fail(GDN_EINVAL, "too many tokens for a launch");
    return GDN_OK;
}
size_t step_part_bytes(const gdn::MlaStepArgs &a) {
    return align_up((size_t)2 * a.units * a.S * a.H * a.dl * 4);
}
size_t step_ml_bytes(const gdn::MlaStepArgs &a) {
    return align_up((size_t)2 * a.units * a.S * a.H * 8);
}

constexpr uint32_t ROPE_FLAGS = GDN_ROPE_NORM | GDN_ROPE_INTERLEAVED;

gdn_status_t check_norm(int64_t M, int32_t H, int32_t d, int32_t r, int32_t dtype, uint32_t flags, float eps) {
    if (M < 0 || H < 1 || d < 1) return fail(GDN_EINVAL, "M must be >= 0, H and d >= 1");
    if (dtype != GDN_F32 && dtype != GDN_BF16) return fail(GDN_EINVAL, "unknown dtype %d", dtype);
    if (flags & ~ROPE_FLAGS) return fail(GDN_EINVAL, "unknown flag bits 0x%x", flags);
    if (d > 512) return fail(GDN_EUNSUPPORTED, "d must be at most 512");
    if (r < 0 || r > d || r % 2) return fail(GDN_EINVAL, "r must be even, in [0, d]");
    if ((flags & GDN_ROPE_NORM) && !(eps > 0.f && isfinite(eps)))
        return fail(GDN_EINVAL, "eps must be positive and finite");
    if ((double)M * H * d >= LIMIT) return fail(GDN_EINVAL, "tensor too large");
    return GDN_OK;
}

} // namespace

extern "C" {

gdn_status_t gdn_mla_fwd(const gdn_mla_shape_t *s, const void *q, const void *k, const void *k_rope, const void *v,
                         const int32_t *lens, void *o, float *lse, void *stream) {
    gdn_status_t st = check_mla(s);
    if (st != GDN_OK) return st;
    const MlaSizes z = mla_sizes(s);
    const Buf b[] = {{q, z.q, "q", 16, false, true},
                     {k, z.k, "k", 16, false, s->Tq > 0},
                     {k_rope, z.kr, "k_rope", 16, false, s->Tq > 0},
                     {v, z.v, "v", 16, false, s->Tq > 0},
                     {lens, z.lens, "lens", 4, false, false},
                     {o, z.o, "o", 16, true, true},
                     {lse, z.lse, "lse", 4, true, false}};
    st = check_bufs(b, 7);
    if (st != GDN_OK) return st;
    if (s->Tq == 0) return ok();
    gdn::MlaFwdArgs a;
    a.s = mla_args(s, q, k, k_rope, v, lens);
    a.o = o;
    a.lse = lse;
    hipStream_t strm = (hipStream_t)stream;
    return hip_status(gdn::bracketed(
                          gdn::K_MLA_FWD,
                          [&] {
                              return s->dtype == GDN_BF16 ? gdn::launch_mla_fwd_bf16(a, strm)
                                                          : gdn::launch_mla_fwd_f32(a, strm);
                          },
                          strm),
                      "gdn_mla_fwd launch");
}

size_t gdn_mla_bwd_workspace_size(const gdn_mla_shape_t *s) {
    if (check_mla(s) != GDN_OK) return 0;
    return mla_delta_bytes(s) + mla_part_bytes(s);
}

gdn_status_t gdn_mla_bwd(const gdn_mla_shape_t *s, const void *q, const void *k, const void *k_rope, const void *v,
                         const int32_t *lens, const void *o, const float *lse, const void *dout, void *dq, void *dk,
                         void *dk_rope, void *dv, void *ws, size_t ws_bytes, void *stream) {
    gdn_status_t st = check_mla(s);
    if (st != GDN_OK) return st;
    const MlaSizes z = mla_sizes(s);
    const size_t need = mla_delta_bytes(s) + mla_part_bytes(s);
    const Buf b[] = {{q, z.q, "q", 16, false, true},          {k, z.k, "k", 16, false, true},
                     {k_rope, z.kr, "k_rope", 16, false, true}, {v, z.v, "v", 16, false, true},
                     {lens, z.lens, "lens", 4, false, false},  {o, z.o, "o", 16, false, true},
                     {lse, z.lse, "lse", 4, false, true},      {dout, z.o, "do", 16, false, true},
                     {dq, z.q, "dq", 16, true, true},          {dk, z.k, "dk", 16, true, true},
                     {dk_rope, z.kr, "dk_rope", 16, true, true}, {dv, z.v, "dv", 16, true, true},
                     {ws, need, "workspace", 1, true, false}};
    st = check_bufs(b, 13);
    if (st != GDN_OK) return st;
    if (need && (!ws || ws_bytes < need))
        return fail(GDN_EWORKSPACE, "gdn_mla_bwd needs %zu bytes of workspace, got %zu", need, ws ? ws_bytes : 0);
    if (need && (uintptr_t)ws % 256) return fail(GDN_EINVAL, "workspace must be 256-byte aligned");
    if (s->Tk == 0) return ok();
    gdn::MlaBwdArgs a;
    a.s = mla_args(s, q, k, k_rope, v, lens);
    a.o = o;
    a.dout = dout;
    a.lse = lse;
    a.delta = (float *)ws;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.dkr = dk_rope;
    a.dkr_part = mla_part_bytes(s) ? (float *)((char *)ws + mla_delta_bytes(s)) : nullptr;
    const bool bf = s->dtype == GDN_BF16;
    hipStream_t strm = (hipStream_t)stream;
    hipError_t e = hipSuccess;
    if (s->Tq > 0) // (no query: the key gradients are zero, which the second kernel writes)
        e = gdn::bracketed(
            gdn::K_MLA_BWD_Q,
            [&] { return bf ? gdn::launch_mla_bwd_q_bf16(a, strm) : gdn::launch_mla_bwd_q_f32(a, strm); }, strm);
    if (e == hipSuccess)
        e = gdn::bracketed(
            gdn::K_MLA_BWD_K,
            [&] { return bf ? gdn::launch_mla_bwd_k_bf16(a, strm) : gdn::launch_mla_bwd_k_f32(a, strm); }, strm);
    if (e == hipSuccess && a.dkr_part)
        e = gdn::bracketed(gdn::K_MLA_ROPE_SUM, [&] { return gdn::launch_mla_rope_sum(a, bf, strm); }, strm);
    return hip_status(e, "gdn_mla_bwd launch");
}

size_t gdn_mla_step_workspace_size(const gdn_mla_step_shape_t *s) {
    if (check_step(s) != GDN_OK) return 0;
    const gdn::MlaStepArgs a = step_args(s);
    return step_part_bytes(a) + step_ml_bytes(a);
}

gdn_status_t gdn_mla_step(const gdn_mla_step_shape_t *s, const void *q, const void *cache, const int32_t *block_table,
                          const int32_t *lens, void *o, float *lse, void *ws, size_t ws_bytes, void *stream) {
    gdn_status_t st = check_step(s);
    if (st != GDN_OK) return st;
    gdn::MlaStepArgs a = step_args(s);
    const size_t e = esize(s->dtype), rows = (size_t)s->N * s->S * s->H, need = step_part_bytes(a) + step_ml_bytes(a);
    const bool some = rows > 0;
    const Buf b[] = {{q, rows * (s->dl + s->dr) * e, "q", 16, false, true},
                     {cache, (size_t)s->pages * s->page_size * (s->dl + s->dr) * e, "cache", 16, false, some},
                     {block_table, (size_t)s->N * s->max_pages * 4, "block_table", 4, false, some},
                     {lens, (size_t)s->N * 4, "lens", 4, false, some},
                     {o, rows * s->dl * e, "o", 16, true, true},
                     {lse, rows * 4, "lse", 4, true, false},
                     {ws, need, "workspace", 1, true, false}};
    st = check_bufs(b, 7);
    if (st != GDN_OK) return st;
    if (!some) return ok();
    if (need && (!ws || ws_bytes < need))
        return fail(GDN_EWORKSPACE, "gdn_mla_step needs %zu bytes of workspace, got %zu", need, ws ? ws_bytes : 0);
    if (need && (uintptr_t)ws % 256) return fail(GDN_EINVAL, "workspace must be 256-byte aligned");
    a.q = q;
    a.cache = cache;
    a.table = block_table;
    a.lens = lens;
    a.o = o;
    a.lse = lse;
    a.part = (float *)ws;
    a.part_ml = (float *)((char *)ws + step_part_bytes(a));
    const bool bf = s->dtype == GDN_BF16;
    hipStream_t strm = (hipStream_t)stream;
    hipError_t he = gdn::bracketed(gdn::K_MLA_STEP, [&] { return gdn::launch_mla_step(a, bf, strm); }, strm);
    if (he == hipSuccess)
        he = gdn::bracketed(gdn::K_MLA_JOIN, [&] { return gdn::launch_mla_join(a, bf, strm); }, strm);
    return hip_status(he, "gdn_mla_step launch");
}

gdn_status_t gdn_norm_rope(int64_t M, int32_t H, int32_t d, int32_t r, int32_t dtype, uint32_t flags, float eps,
                           const void *x, const float *w, const int32_t *positions, const double *freqs, void *y,
                           void *stream) {
    gdn_status_t st = check_norm(M, H, d, r, dtype, flags, eps);
    if (st != GDN_OK) return st;
    const size_t n = (size_t)M * H * d * esize(dtype);
    if (w && !(flags & GDN_ROPE_NORM)) return fail(GDN_EINVAL, "weights need GDN_ROPE_NORM");
    const Buf b[] = {{x, n, "x", 16, false, true},
                     {w, w ? (size_t)d * 4 : 0, "w", 4, false, false},
                     {positions, r > 0 ? (size_t)M * 4 : 0, "positions", 4, false, true},
                     {freqs, r > 0 && M > 0 ? (size_t)r / 2 * 8 : 0, "freqs", 8, false, true},
                     {y, n, "y", 16, true, true}};
    const int same[1][2] = {{0, 4}}; // in place: a row is read whole before it is written
    st = check_bufs(b, 5, same, 1);
    if (st != GDN_OK) return st;
    if (M == 0) return ok();
    gdn::NormRopeArgs a = {};
    a.x = x;
    a.w = w;
    a.pos = positions;
    a.freqs = freqs;
    a.y = y;
    a.M = M;
    a.H = H;
    a.d = d;
    a.r = r;
    a.norm = (flags & GDN_ROPE_NORM) ? 1 : 0;
    a.inter = (flags & GDN_ROPE_INTERLEAVED) ? 1 : 0;
    a.eps = eps;
    hipStream_t strm = (hipStream_t)stream;
    return hip_status(
        gdn::bracketed(gdn::K_NORM_ROPE, [&] { return gdn::launch_norm_rope(a, dtype == GDN_BF16, strm); }, strm),
        "gdn_norm_rope launch");
}

size_t gdn_norm_rope_bwd_workspace_size(int64_t M, int32_t H, int32_t d) {
    if (check_norm(M, H, d, 0, GDN_F32, 0, 0.f) != GDN_OK) return 0;
    return M > 0 ? align_up((size_t)gdn::norm_rope_blocks(M * H, d) * d * 4) : 0;
}

gdn_status_t gdn_norm_rope_bwd(int64_t M, int32_t H, int32_t d, int32_t r, int32_t dtype, uint32_t flags, float eps,
                               const void *dy, const void *x, const float *w, const int32_t *positions,
                               const double *freqs, void *dx, float *dw, void *ws, size_t ws_bytes, void *stream) {
    gdn_status_t st = check_norm(M, H, d, r, dtype, flags, eps);
    if (st != GDN_OK) return st;
    const bool norm = flags & GDN_ROPE_NORM;
    if ((w || dw) && !norm) return fail(GDN_EINVAL, "weights need GDN_ROPE_NORM");
    const size_t n = (size_t)M * H * d * esize(dtype), need = dw ? gdn_norm_rope_bwd_workspace_size(M, H, d) : 0;
    const Buf b[] = {{dy, n, "dy", 16, false, true},
                     {x, norm ? n : 0, "x", 16, false, true},
                     {w, w ? (size_t)d * 4 : 0, "w", 4, false, false},
                     {positions, r > 0 ? (size_t)M * 4 : 0, "positions", 4, false, true},
                     {freqs, r > 0 && M > 0 ? (size_t)r / 2 * 8 : 0, "freqs", 8, false, true},
                     {dx, n, "dx", 16, true, true},
                     {dw, dw ? (size_t)d * 4 : 0, "dw", 4, true, false},
                     {ws, need, "workspace", 1, true, false}};
    st = check_bufs(b, 8);
    if (st != GDN_OK) return st;
    if (need && (!ws || ws_bytes < need))
        return fail(GDN_EWORKSPACE, "gdn_norm_rope_bwd needs %zu bytes of workspace, got %zu", need, ws ? ws_bytes : 0);
    if (need && (uintptr_t)ws % 256) return fail(GDN_EINVAL, "workspace must be 256-byte aligned");
    hipStream_t strm = (hipStream_t)stream;
    if (M == 0) // no row: dw is an empty sum
        return dw ? hip_status(gdn::launch_copy_or_zero(dw, nullptr, d, strm), "gdn_norm_rope_bwd") : ok();
    gdn::NormRopeArgs a = {};
    a.x = x;
    a.dy = dy;
    a.w = w;
    a.pos = positions;
    a.freqs = freqs;
    a.y = dx;
    a.dw = dw;
    a.dw_part = (float *)ws;
    a.M = M;
    a.H = H;
    a.d = d;
    a.r = r;
    a.norm = norm ? 1 : 0;
    a.inter = (flags & GDN_ROPE_INTERLEAVED) ? 1 : 0;
    a.eps = eps;
    a.nblk = gdn::norm_rope_blocks(M * H, d);
    hipError_t e = gdn::bracketed(
        gdn::K_NORM_ROPE_BWD, [&] { return gdn::launch_norm_rope_bwd(a, dtype == GDN_BF16, strm); }, strm);
    if (e == hipSuccess && dw)
        e = gdn::bracketed(gdn::K_NORM_SUM, [&] { return gdn::launch_norm_sum(a, strm); }, strm);
    return hip_status(e, "gdn_norm_rope_bwd launch");
}

gdn_status_t gdn_mla_write(int64_t n, int32_t dl, int32_t dr, int32_t dtype, uint32_t flags, float eps, const void *c,
                           const void *k_rope, const float *w, const int32_t *positions, const double *freqs,
                           const int32_t *slots, void *cache, int64_t n_slots, void *stream) {
    if (n < 0 || dl < 1 || dr < 0) return fail(GDN_EINVAL, "n, dr must be >= 0 and dl >= 1");
    if (dtype != GDN_F32 && dtype != GDN_BF16) return fail(GDN_EINVAL, "unknown dtype %d", dtype);
    if (flags & ~ROPE_FLAGS) return fail(GDN_EINVAL, "unknown flag bits 0x%x", flags);
    if (dl % 8 || dl > 512 || dr % 8 || dr > 64)
        return fail(GDN_EUNSUPPORTED, "dl must be a multiple of 8 up to 512, dr one up to 64");
    const bool norm = flags & GDN_ROPE_NORM;
    if (norm && !(eps > 0.f && isfinite(eps))) return fail(GDN_EINVAL, "eps must be positive and finite");
    if (w && !norm) return fail(GDN_EINVAL, "weights need GDN_ROPE_NORM");
    if (n_slots < 0 || (double)n_slots >= LIMIT || (double)n * (dl + dr) >= LIMIT)
        return fail(GDN_EINVAL, "tokens or cache too large");
    const size_t e = esize(dtype), N = (size_t)n;
    const bool turn = dr > 0 && freqs;
    if (turn && N && !positions) return fail(GDN_EINVAL, "positions is NULL");
    const Buf b[] = {{c, N * dl * e, "c", 16, false, true},
                     {k_rope, N * dr * e, "k_rope", 4, false, true},
                     {w, w ? (size_t)dl * 4 : 0, "w", 4, false, false},
                     {positions, turn ? N * 4 : 0, "positions", 4, false, false},
                     {freqs, turn ? (size_t)dr / 2 * 8 : 0, "freqs", 8, false, false},
                     {slots, N * 4, "slots", 4, false, true},
                     {cache, (size_t)n_slots * (dl + dr) * e, "cache", 16, true, true}};
    const gdn_status_t st = check_bufs(b, 7);
    if (st != GDN_OK) return st;
    if (n == 0 || n_slots == 0) return ok();
    gdn::MlaWriteArgs a;
    a.c = c;
    a.kr = k_rope;
    a.w = w;
    a.pos = positions;
    a.slots = slots;
    a.freqs = turn ? freqs : nullptr;
    a.cache = cache;
    a.n_slots = n_slots;
    a.n = (int)n;
    a.dl = dl;
    a.dr = dr;
    a.norm = norm ? 1 : 0;
    a.inter = (flags & GDN_ROPE_INTERLEAVED) ? 1 : 0;
    a.eps = eps;
    hipStream_t strm = (hipStream_t)stream;
    return hip_status(
        gdn::bracketed(gdn::K_MLA_WRITE, [&] { return gdn::launch_mla_write(a, dtype == GDN_BF16, strm); }, strm),
        "gdn_mla_write launch");
}

gdn_status_t gdn_page_plan(int32_t N, int32_t max_pages, int32_t n_pages, int32_t page_size, int32_t max_tokens,
                           const int32_t *lens, const int32_t *new_lens, int32_t *block_table, int32_t *free_pages,
                           const int32_t *n_free, int32_t *lens_out, int32_t *n_free_out, int32_t *granted,
                           int32_t *starts, int32_t *slots, int32_t *positions, void *stream) {
    if (N < 0 || max_pages < 1 || n_pages < 1 || page_size < 1 || max_tokens < 0)
        return fail(GDN_EINVAL, "N, max_tokens must be >= 0, max_pages, n_pages and page_size >= 1");
    if ((double)N * max_pages > LIMIT - AHEAD || max_tokens > 2147483647 - 255)
        return fail(GDN_EINVAL, "table or token count too large");
    const size_t n = (size_t)N * 4;
    const Buf b[] = {{lens, n, "lens", 4, false, true},
                     {new_lens, n, "new_lens", 4, false, true},
                     {n_free, 4, "n_free", 4, false, true},
                     {block_table, n * max_pages, "block_table", 4, true, true},
                     {free_pages, (size_t)n_pages * 4, "free_pages", 4, true, true},
                     {lens_out, n, "lens_out", 4, true, true},
                     {n_free_out, 4, "n_free_out", 4, true, true},
                     {granted, n, "granted", 4, true, true},
                     {starts, n + 4, "starts", 4, true, true},
                     {slots, (size_t)max_tokens * 4, "slots", 4, true, true},
                     {positions, (size_t)max_tokens * 4, "positions", 4, true, true}};
    const int same[2][2] = {{0, 5}, {2, 6}};
    const gdn_status_t st = check_bufs(b, 11, same, 2);
    if (st != GDN_OK) return st;
    gdn::PagePlanArgs a;
    a.lens = lens;
    a.fresh = new_lens;
    a.table = block_table;
    a.stack = free_pages;
    a.n_free = n_free;
    a.lens_out = lens_out;
    a.n_free_out = n_free_out;
    a.granted = granted;
    a.starts = starts;
    a.slots = slots;
    a.positions = positions;
    a.N = N;
    a.cols = max_pages;
    a.F = n_pages;
    a.page = page_size;
    a.cap = max_tokens;
    hipStream_t strm = (hipStream_t)stream;
    hipError_t e = gdn::bracketed(gdn::K_PAGE_PLAN, [&] { return gdn::launch_page_plan(a, strm); }, strm);
    if (e == hipSuccess && gdn::page_fill_separate(max_tokens))
        e = gdn::bracketed(gdn::K_PAGE_FILL, [&] { return gdn::launch_page_fill(a, strm); }, strm);
    return hip_status(e, "gdn_page_plan launch");
}

} // extern "C"
