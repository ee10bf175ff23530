// Block tables and slot maps of the paged cache, built on the GPU.
//
// page_plan_kernel, one workgroup: sequences that ended push their pages back
// on the free stack; then, in order, every sequence that still has room in its
// table row gets its new tokens while tokens (cap) and free pages last, its
// new pages popped from the stack's top into its row. All of it is prefix sums
// over the sequences (a thousand at a time), and the page moves are spread
// over the threads by a binary search in those sums, so no thread walks a long
// sequence alone. The sums are whole numbers: the result does not depend on
// any order. page_fill gives every new token its position and slot by a search
// in `starts`; a small batch does it in the same launch, since there the call
// is bound by launch latency (a few microseconds) and not by its bytes.
#include "gdn_mla.hpp"

namespace gdn {

constexpr int PL = 1024; // threads, and sequences per step
constexpr int FILL_ONE = 4096;

// Inclusive prefix sum over the workgroup; `total` is the sum of all.
template <class T> __device__ __forceinline__ T scan(T x, T *waves, T &total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const T y = __shfl_up(x, o, 64);
        if (lane >= o) x += y;
    }
    __syncthreads(); // (the previous scan's reads of waves are done)
    if (lane == 63) waves[wave] = x;
    __syncthreads();
    T before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < PL / 64; ++w) {
        before += w < wave ? waves[w] : T(0);
        total += waves[w];
    }
    return x + before;
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

// Position and slot of new token t.
__device__ __forceinline__ void fill_token(const PagePlanArgs &a, int t) {
    int slot = -1, pos = 0;
    if (t < a.starts[a.N]) {
        const int i = owner(a.starts + 1, a.N, t);
        pos = a.lens_out[i] - a.granted[i] + (t - a.starts[i]);
        const int id = a.table[(size_t)i * a.cols + pos / a.page];
        const long long s = (long long)id * a.page + pos % a.page;
        slot = id < 0 || s > 2147483647LL ? -1 : (int)s;
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
}

__global__ __launch_bounds__(PL) void page_plan_kernel(PagePlanArgs a, int fill) {
    __shared__ int ends[PL], held_s[PL];
    __shared__ int wi[PL / 64];
    __shared__ long long wl[PL / 64];
    const int tid = threadIdx.x, page = a.page;
    const int room = (int)min((long long)a.cols * page, 2147483647LL); // tokens a table row holds
    int top = min(max(*a.n_free, 0), a.F);
    // ended sequences: pages back on the stack
    for (int c = 0; c < a.N; c += PL) {
        const int i = c + tid;
        const bool gone = i < a.N && a.fresh[i] < 0;
        const int len = gone ? min(max(a.lens[i], 0), room) : 0;
        const int back = len / page + (len % page != 0);
        int total;
        ends[tid] = scan(back, wi, total);
        held_s[tid] = back;
        __syncthreads();
        for (int k = tid; k < total; k += PL) {
            const int o = owner(ends, PL, k), col = k - (ends[o] - held_s[o]);
            if (k < a.F - top) a.stack[top + k] = a.table[(size_t)(c + o) * a.cols + col];
        }
        top = min((long long)top + total, (long long)a.F);
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
        const int held = len / page + (len % page != 0);
        const long long end = (long long)len + max(fresh, 0);
        const bool fits = end <= room;
        const int ask = fits ? max(fresh, 0) : 0;
        const int need = ask > 0 ? (int)((end + page - 1) / page) - held : 0;
        int np, ns, nu;
        long long na;
        const int need_end = pages_before + scan(need, wi, np);
        const long long ask_end = asked_before + scan((long long)ask, wl, na);
        const bool yes = fits && ask_end <= a.cap && (need == 0 || need_end <= top);
        const int granted = yes ? ask : 0, used = yes ? need : 0;
        const int start_end = starts_before + scan(granted, wi, ns);
        ends[tid] = scan(used, wi, nu);
        held_s[tid] = held - (ends[tid] - used); // first new column, less the pages before this sequence's
        if (live) {
            a.granted[i] = granted;
            a.lens_out[i] = fresh < 0 ? 0 : len + granted;
            a.starts[i + 1] = start_end;
        }
        __syncthreads();
        for (int k = tid; k < nu; k += PL) {
            const int o = owner(ends, PL, k);
            a.table[(size_t)(c + o) * a.cols + held_s[o] + k] = a.stack[top - 1 - used_before - k];
        }
        pages_before += np;
        asked_before += na;
        starts_before += ns;
        used_before += nu;
        __syncthreads();
    }
    if (tid == 0) *a.n_free_out = top - used_before;
    if (!fill) return;
    for (int t = tid; t < a.cap; t += PL) fill_token(a, t);
}

__global__ __launch_bounds__(256) void page_fill_kernel(PagePlanArgs a) {
    const int t = blockIdx.x * 256 + threadIdx.x;
    if (t < a.cap) fill_token(a, t);
}

bool page_fill_separate(int cap) { return cap > FILL_ONE; }

hipError_t launch_page_plan(const PagePlanArgs &a, hipStream_t st) {
    hipLaunchKernelGGL(page_plan_kernel, dim3(1), dim3(PL), 0, st, a, page_fill_separate(a.cap) ? 0 : 1);
    return hipGetLastError();
}
hipError_t launch_page_fill(const PagePlanArgs &a, hipStream_t st) {
    hipLaunchKernelGGL(page_fill_kernel, dim3((unsigned)((a.cap + 255) / 256)), dim3(256), 0, st, a);
    return hipGetLastError();
}

} // namespace gdn
