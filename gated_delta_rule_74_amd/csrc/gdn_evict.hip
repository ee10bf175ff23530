// Eviction of cached rows by weight: which rows a sequence keeps, and their
// move to the front of its pages.
//
// choose, one workgroup per sequence: the weight of the lightest row kept is
// found digit by digit, eleven, eleven and ten bits of the weights' ordered bit patterns at a
// time, each from a histogram in LDS of the rows that agree in the digits
// before (whole numbers: no order changes them). A last pass counts, for every
// segment of the sequence, the rows above that weight and of exactly that weight, and
// prefix sums of those tell every segment where its rows go and how many of
// the equal ones come before it.
//
// move, one workgroup per segment: reads its kept rows into registers, and
// writes them to the front once every segment that still holds rows in their new places
// has been read. Bytes bound it: each kept row is read and written once, in place. A
// segment goes by the ticket that its workgroup draws from its sequence's
// counter and waits for segments of lower tickets alone. Those
// workgroups are running, and set their flag before they wait for anything, so every wait ends.
#include "gdn_serve.hpp"

namespace gdn {

constexpr int ET = 1024; // threads of both kernels

constexpr int EV = 18;   // 16-byte pieces a thread holds: a segment's rows
static_assert(evict_segment(72) * 72 <= ET * EV && evict_segment(EVICT_ROW16) * EVICT_ROW16 <= ET * EV, "a segment fits");

// The order of the weights as unsigned numbers: NaN above all, -0 as 0; 0 is left for rows outside the pool.
__device__ __forceinline__ uint32_t key_of(float w) {
    if (w != w) return 0xffffffffu;
    const uint32_t b = __float_as_uint(w + 0.f);
    return b >> 31 ? ~b : b | 0x80000000u; // (at least ~0xff800000, -inf's)
}
struct Lot { // what a sequence keeps
    int n, k, a, b; // rows, rows kept, first and last ones kept in any case
};
__device__ __forceinline__ Lot lot_of(const EvictArgs &e, int i) {
    Lot s;
    s.n = (int)min((long long)max(e.lens[i], 0), (long long)e.cols * e.page);
    s.k = min(max(e.keep[i], 0), s.n);
    s.a = min(e.first, s.k);
    s.b = min(e.recent, s.k - s.a);
    return s;
}
// slot of a row, -1: its table entry lies outside the pool
__device__ __forceinline__ int slot_of(const EvictArgs &e, const int *tb, int pos) {
    const int entry = tb[(unsigned)pos / (unsigned)e.page];
    return (unsigned)entry < (unsigned)e.pages ? entry * e.page + (int)((unsigned)pos % (unsigned)e.page) : -1;
}
__device__ __forceinline__ uint32_t row_key(const EvictArgs &e, const int *tb, int pos) {
    const int s = slot_of(e, tb, pos);
    return s < 0 ? 0u : key_of(e.weights[s]);
}

__global__ __launch_bounds__(ET) void evict_choose_kernel(EvictArgs e) {
    __shared__ int hist[2048];
    __shared__ int waves[ET / 64][2];
    __shared__ int pick[2]; // the digit, and the rows above it
    const int n = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const Lot s = lot_of(e, n);
    const int seg = evict_segment(e.row16), nseg = (s.n + seg - 1) / seg;
    if (tid == 0) {
        e.lens_out[n] = s.k;
        e.ticket[n] = 0;
    }
    if (s.k == s.n) return; // (the move leaves such a sequence alone too)
    int *done = e.done + (size_t)n * e.segs;
    for (int i = tid; i < nseg; i += ET) done[i] = 0;
    const int *tb = e.table + (size_t)n * e.cols;
    const int lo = s.a, hi = s.n - s.b; // the rows to choose among
    int want = s.k - s.a - s.b;         // of which so many stay
    // the key of the lightest that stays: digit by digit, the largest with enough rows at or above it
    uint32_t prefix = 0;
    if (want > 0) {
        for (int shift = 21; shift >= 0; shift = shift == 21 ? 10 : shift == 10 ? 0 : -1) {
            const int bits = shift ? 11 : 10, above = shift + bits;
            for (int i = tid; i < 2048; i += ET) hist[i] = 0;
            __syncthreads();
            for (int p = lo + tid; p < hi; p += ET) {
                const uint32_t key = row_key(e, tb, p);
                if (above == 32 || key >> above == prefix >> above) atomicAdd(&hist[key >> shift & ((1u << bits) - 1)], 1);
            }
            __syncthreads();
            // suffix sums: thread t owns digits 2t and 2t + 1 from the top
            const int top = (1 << bits) - 1, d0 = top - 2 * tid, h0 = d0 >= 0 ? hist[d0] : 0, h1 = d0 >= 1 ? hist[d0 - 1] : 0;
            int x = h0 + h1;
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const int y = __shfl_up(x, o, 64);
                if (lane >= o) x += y;
            }
            if (lane == 63) waves[wave][0] = x;
            __syncthreads();
            for (int w = 0; w < wave; ++w) x += waves[w][0];
            const int before = x - h0 - h1; // rows above digit d0
            if (d0 >= 0 && before < want && before + h0 >= want) {
                pick[0] = d0;
                pick[1] = before;
            }
            if (d0 >= 1 && before + h0 < want && x >= want) {
                pick[0] = d0 - 1;
                pick[1] = before + h0;
            }
            __syncthreads();
            prefix |= (uint32_t)pick[0] << shift;
            want -= pick[1];
            __syncthreads();
        }
    } else {
        prefix = 0xffffffffu; // none of the middle: equal ones (NaN) come to none
    }
    const uint32_t bar = prefix;
    const int spare = want;
    if (tid == 0) {
        e.bar[n] = bar;
        e.spare[n] = spare;
    }
    // kept for sure, and of the bar's weight, per segment: a wave counts one after the other
    int *kept = e.kept + (size_t)n * e.segs, *ties = e.ties + (size_t)n * e.segs;
    for (int g = wave; g < nseg; g += ET / 64) {
        int more = 0, same = 0;
        for (int j = 0; j < seg; j += 64) {
            const int p = g * seg + j + lane;
            const bool in = p < s.n, sure = in && (p < lo || p >= hi), mid = in && !sure;
            const uint32_t key = mid ? row_key(e, tb, p) : 0u;
            more += __popcll(__ballot(sure || (mid && key > bar)));
            same += __popcll(__ballot(mid && key == bar));
        }
        if (lane == 0) {
            kept[g] = more;
            ties[g] = same;
        }
    }
    __syncthreads();
    // their prefix sums; of the equal ones the first `spare` stay
    int more0 = 0, same0 = 0;
    for (int g0 = 0; g0 < nseg; g0 += ET) {
        const int g = g0 + tid;
        const int m0 = g < nseg ? kept[g] : 0, t0 = g < nseg ? ties[g] : 0;
        int m = m0, t = t0;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int y = __shfl_up(m, o, 64), z = __shfl_up(t, o, 64);
            if (lane >= o) {
                m += y;
                t += z;
            }
        }
        __syncthreads(); // (the last round's readers are done)
        if (lane == 63) {
            waves[wave][0] = m;
            waves[wave][1] = t;
        }
        __syncthreads();
        int mall = 0, tall = 0;
        for (int w = 0; w < ET / 64; ++w) {
            if (w < wave) {
                m += waves[w][0];
                t += waves[w][1];
            }
            mall += waves[w][0];
            tall += waves[w][1];
        }
        if (g < nseg) {
            const int eq = same0 + t - t0; // equal ones before the segment
            ties[g] = eq;
            kept[g] = more0 + m - m0 + min(eq, spare);
        }
        more0 += mall;
        same0 += tall;
    }
}

__global__ __launch_bounds__(ET) void evict_move_kernel(EvictArgs e) {
    __shared__ int from[256], to[256];
    __shared__ int counts[4][2], drawn, all;
    const int n = blockIdx.x / e.segs, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const Lot s = lot_of(e, n);
    if (s.k == s.n) return;
    const int seg = evict_segment(e.row16), nseg = (s.n + seg - 1) / seg;
    if ((int)(blockIdx.x % e.segs) >= nseg) return; // as many workgroups as the sequence has segments draw tickets
    if (tid == 0) drawn = atomicAdd(&e.ticket[n], 1);
    __syncthreads();
    const int g = drawn;
    const int *tb = e.table + (size_t)n * e.cols;
    int *done = e.done + (size_t)n * e.segs;
    const uint32_t bar = e.bar[n];
    const int spare = e.spare[n], base = e.kept[(size_t)n * e.segs + g], ties = e.ties[(size_t)n * e.segs + g];
    // which rows stay, and where they go
    bool stay = false;
    int slot = -1, rank = 0, same = 0;
    float weight = 0.f;
    if (tid < seg) {
        const int p = g * seg + tid;
        bool sure = false, tie = false;
        if (p < s.n) {
            slot = slot_of(e, tb, p);
            weight = slot < 0 ? 0.f : e.weights[slot];
            const uint32_t key = slot < 0 ? 0u : key_of(weight);
            const bool mid = p >= s.a && p < s.n - s.b;
            sure = !mid || key > bar;
            tie = mid && key == bar;
        }
        const uint64_t eq = __ballot(tie), below = (1ull << lane) - 1;
        same = __popcll(eq & below);
        if (lane == 0) counts[wave][0] = __popcll(eq);
        stay = sure;
        rank = tie ? 1 : 0;
    }
    __syncthreads();
    if (tid < seg) {
        for (int w = 0; w < wave; ++w) same += counts[w][0];
        if (rank && ties + same < spare) stay = true;
        const uint64_t st = __ballot(stay), below = (1ull << lane) - 1;
        rank = __popcll(st & below);
        if (lane == 0) counts[wave][1] = __popcll(st);
    }
    __syncthreads();
    if (tid < seg) {
        for (int w = 0; w < wave; ++w) rank += counts[w][1];
        if (stay) {
            from[rank] = slot;
            to[rank] = slot_of(e, tb, base + rank);
        }
        if (tid == seg - 1) all = rank + (stay ? 1 : 0);
    }
    __syncthreads();
    const int count = all, row16 = e.row16, pieces = count * row16;
    // the rows, into registers (a segment whose rows all stay where they are has nothing to read)
    const bool moves = count > 0 && base < g * seg + min(seg, s.n - g * seg) - count;
    u32x4 x[EV];
    u32x4 *pool = (u32x4 *)e.cache;
    if (moves) {
#pragma unroll
        for (int v = 0; v < EV; ++v) {
            if (v * ET >= pieces) continue;
            const int i = min(tid + v * ET, pieces - 1), row = (unsigned)i / (unsigned)row16;
            const int src = from[row];
            x[v] = load16(src < 0 ? (const void *)&mla_zeros
                                  : (const void *)(pool + (size_t)(unsigned)src * row16 + (i - row * row16)));
        }
    }
    // all of it is here before the flag says so
    wait_vmem();
    __syncthreads();
    if (tid == 0) __hip_atomic_store(&done[g], 1, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_AGENT);
    if (!moves) return;
    // the rows' new places hold rows of at most two or three segments before this one
    if (tid == 0) {
        const int g0 = base / seg, g1 = min((base + count - 1) / seg, g - 1);
        for (int i = g0; i <= g1; ++i)
            while (!__hip_atomic_load(&done[i], __ATOMIC_ACQUIRE, __HIP_MEMORY_SCOPE_AGENT)) __builtin_amdgcn_s_sleep(2);
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < EV; ++v) {
        const int i = tid + v * ET, row = (unsigned)i / (unsigned)row16;
        if (i < pieces && from[row] >= 0 && to[row] >= 0) pool[(size_t)(unsigned)to[row] * row16 + (i - row * row16)] = x[v];
    }
    if (stay && slot >= 0) {
        const int dst = to[rank];
        if (dst >= 0) e.weights[dst] = weight;
    }
}

hipError_t launch_evict_choose(const EvictArgs &a, hipStream_t st) {
    hipLaunchKernelGGL(evict_choose_kernel, dim3(a.N), dim3(ET), 0, st, a);
    return hipGetLastError();
}
hipError_t launch_evict_move(const EvictArgs &a, hipStream_t st) {
    hipLaunchKernelGGL(evict_move_kernel, dim3((unsigned)((long long)a.N * a.segs)), dim3(ET), 0, st, a);
    return hipGetLastError();
}

} // namespace gdn
