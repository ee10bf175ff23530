// Block tables and slot maps of the paged cache, built on the GPU.
//
// page_plan_kernel, one workgroup: sequences that ended push their pages back
// on the free stack; then, in order, every sequence that still has room in its
// table row gets its new tokens while tokens (cap) and free pages last, its
// new pages popped from the stack's top into its row. All of it is prefix sums
// over the sequences (a thousand at a time), and the page moves are spread
// over the threads by a binary search in those sums, so no thread walks a long
// sequence alone. The sums are whole numbers: the result does not depend on
// any order. A small batch gives its new tokens their positions and slots in
// the same launch, since there the call is bound by the launch and the chain of
// sums (256 sequences: 8 us); with more tokens than FILL_ONE a second launch does that, and
// the moves of new pages with it, over the whole chip (1024 prompts of 400
// tokens, 26000 pages: 39 us in one workgroup, 16 + 13 us so).
#include "gdn_mla.hpp"

namespace gdn {

constexpr int PL = 1024; // threads, and sequences per step
constexpr int FILL_ONE = 4096;

// Inclusive prefix sums of K values at once over a workgroup of NT threads;
// total: the sums of all.
template <int NT, int K, class T> __device__ __forceinline__ void scan(T (&x)[K], T (*waves)[K], T (&total)[K]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const T y = __shfl_up(x[k], o, 64);
            if (lane >= o) x[k] += y;
        }
    }
    __syncthreads(); // (the previous scan's reads of waves are done)
    if (lane == 63) {
#pragma unroll
        for (int k = 0; k < K; ++k) waves[wave][k] = x[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        T before = 0;
        total[k] = 0;
#pragma unroll
        for (int w = 0; w < NT / 64; ++w) {
            const T y = waves[w][k];
            before += w < wave ? y : T(0);
            total[k] += y;
        }
        x[k] += before;
    }
}

// First i < n with ends[i] > x (n - 1 when there is none).
__device__ __forceinline__ int owner(const int *ends, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (ends[mid] > x) hi = mid;
        else lo = mid + 1;
    }
    return lo;
}

__device__ __forceinline__ int pages_of(int tokens, int page) { return tokens / page + (tokens % page != 0); }

// A new token's position and slot, given its sequence, position and page.
__device__ __forceinline__ void put_token(const PagePlanArgs &a, int t, int pos, int id) {
    const long long s = (long long)id * a.page + pos % a.page;
    a.slots[t] = id < 0 || s > 2147483647LL ? -1 : (int)s;
    a.positions[t] = pos;
}

__global__ __launch_bounds__(PL) void page_plan_kernel(PagePlanArgs a, int fill) {
    __shared__ int ends[PL], held_s[PL];
    __shared__ int w1[PL / 64][1], w2[PL / 64][2];
    __shared__ long long wl[PL / 64][2];
    const int tid = threadIdx.x, page = a.page;
    const int room = (int)min((long long)a.cols * page, 2147483647LL); // tokens a table row holds
    int top = min(max(*a.n_free, 0), a.F);
    // ended sequences: pages back on the stack
    for (int c = 0; c < a.N; c += PL) {
        const int i = c + tid;
        const bool gone = i < a.N && a.fresh[i] < 0;
        if (!__syncthreads_or(gone)) continue;
        const int back = gone ? pages_of(min(max(a.lens[i], 0), room), page) : 0;
        int x[1] = {back}, total[1];
        scan<PL>(x, w1, total);
        ends[tid] = x[0];
        held_s[tid] = back;
        __syncthreads();
        // a run of pages to each thread: one search, then step by step
        const int run = (total[0] + PL - 1) / PL, k0 = tid * run, k1 = min(k0 + run, total[0]);
        for (int k = k0, o = k0 < k1 ? owner(ends, PL, k0) : 0; k < k1; ++k) {
            while (ends[o] <= k) ++o;
            if (k < a.F - top) a.stack[top + k] = a.table[(size_t)(c + o) * a.cols + k - (ends[o] - held_s[o])];
        }
        top = (int)min((long long)top + total[0], (long long)a.F);
        __syncthreads();
    }
    // who gets the tokens asked for, and the pages for them
    int pages_before = 0, starts_before = 0, used_before = 0;
    long long asked_before = 0;
    if (tid == 0) a.starts[0] = 0;
    for (int c = 0; c < a.N; c += PL) {
        const int i = c + tid;
        const bool live = i < a.N;
        const int fresh = live ? a.fresh[i] : 0;
        const int len = live ? min(max(a.lens[i], 0), room) : 0;
        const int held = pages_of(len, page);
        const long long end = (long long)len + max(fresh, 0);
        const bool fits = end <= room;
        const int ask = fits ? max(fresh, 0) : 0;
        const int need = ask > 0 ? (int)((end + page - 1) / page) - held : 0;
        long long q[2] = {need, ask}, qt[2];
        scan<PL>(q, wl, qt);
        const bool yes = fits && asked_before + q[1] <= a.cap && (need == 0 || pages_before + q[0] <= top);
        const int granted = yes ? ask : 0, used = yes ? need : 0;
        int g[2] = {granted, used}, gt[2];
        scan<PL>(g, w2, gt);
        if (live) {
            a.granted[i] = granted;
            a.lens_out[i] = fresh < 0 ? 0 : len + granted;
            a.starts[i + 1] = starts_before + g[0];
        }
        if (fill && gt[1] > 0) { // (else the slots' launch moves the pages)
            ends[tid] = g[1];
            held_s[tid] = held - (g[1] - used); // first new column, less the pages before this sequence's
            __syncthreads();
            for (int k = tid; k < gt[1]; k += PL) {
                const int o = owner(ends, PL, k);
                a.table[(size_t)(c + o) * a.cols + held_s[o] + k] = a.stack[top - 1 - used_before - k];
            }
        }
        pages_before += (int)qt[0];
        asked_before += qt[1];
        starts_before += gt[0];
        used_before += gt[1];
        __syncthreads();
    }
    if (tid == 0) *a.n_free_out = top - used_before;
    if (!fill) return;
    for (int t = tid; t < a.cap; t += PL) {
        if (t >= starts_before) {
            a.slots[t] = -1;
            a.positions[t] = 0;
            continue;
        }
        const int i = owner(a.starts + 1, a.N, t);
        const int pos = a.lens_out[i] - a.granted[i] + (t - a.starts[i]);
        put_token(a, t, pos, a.table[(size_t)i * a.cols + pos / page]);
    }
}

// Many new tokens: 256 of them to a workgroup. It sums the pages taken by the
// sequences before its first token (and by all: that is where the stack's top
// was), and by the ones that begin in it, so a token knows its page's place on
// the stack; a page's first token, always a new one, puts it into the table.
constexpr int FT = 256;
__global__ __launch_bounds__(FT) void page_fill_kernel(PagePlanArgs a) {
    __shared__ int waves[FT / 64][2];
    const int t0 = blockIdx.x * FT, t = t0 + threadIdx.x, total = a.starts[a.N], page = a.page;
    if (t0 >= total) {
        if (t < a.cap) {
            a.slots[t] = -1;
            a.positions[t] = 0;
        }
        return;
    }
    const int first = owner(a.starts + 1, a.N, t0); // sequence of the first token
    int sum[2] = {0, 0}, all[2];                    // pages taken before it, by all
    for (int i = threadIdx.x; i < a.N; i += FT) {
        const int n = a.lens_out[i], taken = pages_of(n, page) - pages_of(n - a.granted[i], page);
        if (i < first) sum[0] += taken;
        sum[1] += taken;
    }
    scan<FT>(sum, waves, all);
    const int before = all[0], top = *a.n_free_out + all[1];
    int i = first, pos = 0, held = 0, own = 0;
    const bool live = t < total;
    if (live) {
        i = owner(a.starts + 1, a.N, t);
        const int n = a.lens_out[i], g = a.granted[i];
        pos = n - g + (t - a.starts[i]);
        held = pages_of(n - g, page);
        own = pages_of(n, page) - held;
    }
    // pages of the sequences up to this token's own, of those that begin here
    int x[2] = {live && t == a.starts[i] && i != first ? own : 0, live && i == first && threadIdx.x == 0 ? own : 0}, xt[2];
    const int mine = own;
    scan<FT>(x, waves, xt);
    if (!live) {
        if (t < a.cap) {
            a.slots[t] = -1;
            a.positions[t] = 0;
        }
        return;
    }
    const int prefix = before + (i == first ? 0 : xt[1] + x[0] - mine);
    const int col = pos / page;
    int *entry = a.table + (size_t)i * a.cols + col;
    int id;
    if (col < held) {
        id = *entry;
    } else {
        id = a.stack[top - 1 - (prefix + col - held)];
        if (pos % page == 0) *entry = id;
    }
    put_token(a, t, pos, id);
}

bool page_fill_separate(int cap) { return cap > FILL_ONE; }

hipError_t launch_page_plan(const PagePlanArgs &a, hipStream_t st) {
    hipLaunchKernelGGL(page_plan_kernel, dim3(1), dim3(PL), 0, st, a, page_fill_separate(a.cap) ? 0 : 1);
    return hipGetLastError();
}
hipError_t launch_page_fill(const PagePlanArgs &a, hipStream_t st) {
    hipLaunchKernelGGL(page_fill_kernel, dim3((unsigned)((a.cap + FT - 1) / FT)), dim3(FT), 0, st, a);
    return hipGetLastError();
}

} // namespace gdn
