// Eviction of cached rows by weight: which rows a sequence keeps, and their
// move to the front of its pages.
//
// choose: the weight of the lightest row kept is found digit by digit, eleven,
// eleven and ten bits of the weights' ordered bit patterns at a time, each from
// a histogram of the rows that agree in the digits before (whole numbers: no
// order changes them). Then every segment of the sequence counts its rows above that
// weight and of exactly that weight, and prefix sums of those tell a segment
// where its rows go and how many of the equal ones come before it. A sequence
// of up to 32768 rows is one workgroup's, which holds the weights in registers
// throughout; longer ones are cut into chunks, a launch to a digit, each
// workgroup adding up its sequence's histograms of the digit before for itself (131072
// rows: 270 us in one workgroup that read the weights again for every digit).
//
// move: a workgroup reads the kept rows of a segment into registers, and
// writes them to the front once every segment that still holds rows in their
// new places has been read. Bytes bound it: each kept row is read and written once, in
// place. A segment goes by the ticket that its workgroup draws from its
// sequence's counter and waits for segments of lower tickets alone. Those were
// drawn before it, by workgroups that are running, which take their tickets in the order they drew them and
// set a segment's flag before they wait for anything on its account: a wait
// leads only to earlier draws, so every wait ends. The next segment's ticket and choice are requested
// while this one's rows are on their way (256 sequences of up to 4096 rows of 160 bf16: 57 us one after the other, 45
// so, 3.8 TB/s read and written; one of 131072 rows of 576: 53 us, 2.8 TB/s; a large copy makes 4.8).
#include "gdn_serve.hpp"

namespace gdn {

constexpr int ET = 1024, EM = EVICT_MOVE; // threads of the two kernels
constexpr int EV = EVICT_HELD;
static_assert(evict_segment(EVICT_ROW16) * EVICT_ROW16 <= EM * EV && evict_segment(1) <= EM, "a segment fits");

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
// segments of a sequence that gives up rows
__device__ __forceinline__ int move_segments(const EvictArgs &e, int i, int seg) {
    const Lot s = lot_of(e, i);
    return s.k == s.n ? 0 : (s.n + seg - 1) / seg;
}
// slot of a row, -1: its table entry lies outside the pool
__device__ __forceinline__ int slot_in(const EvictArgs &e, int entry, int pos) {
    return (unsigned)entry < (unsigned)e.pages ? entry * e.page + (int)((unsigned)pos % (unsigned)e.page) : -1;
}

// The digits of a key, from the top.
__device__ __forceinline__ int digit_shift(int i) { return i == 0 ? 21 : i == 1 ? 10 : 0; }
__device__ __forceinline__ int digit_bits(int i) { return i == 2 ? 10 : 11; }

// Keys of KR * ET rows from `base` on, every ET-th one to a thread (so a wave holds 64 rows that follow each other).
template <int KR> struct Keys {
    uint32_t k[KR];
    __device__ __forceinline__ void load(const EvictArgs &e, const int *tb, int base, const Lot &s) {
        constexpr int B = KR < 8 ? KR : 8; // requested together
#pragma unroll
        for (int u0 = 0; u0 < KR; u0 += B) {
            if (base + u0 * ET >= s.n) break;
            int at[B];
            float w[B];
#pragma unroll
            for (int u = 0; u < B; ++u)
                at[u] = tb[(unsigned)min(base + (u0 + u) * ET + (int)threadIdx.x, s.n - 1) / (unsigned)e.page];
#pragma unroll
            for (int u = 0; u < B; ++u) {
                at[u] = slot_in(e, at[u], min(base + (u0 + u) * ET + (int)threadIdx.x, s.n - 1));
                w[u] = e.weights[max(at[u], 0)];
            }
#pragma unroll
            for (int u = 0; u < B; ++u) k[u0 + u] = at[u] < 0 ? 0u : key_of(w[u]);
        }
    }
    // rows to choose among that agree with `prefix` in the digits before the i-th, by that digit
    __device__ __forceinline__ void count(int *hist, int base, const Lot &s, uint32_t prefix, int i) const {
        const int shift = digit_shift(i), above = shift + digit_bits(i);
#pragma unroll
        for (int u = 0; u < KR; ++u) {
            if (base + u * ET >= s.n) break;
            const int p = base + u * ET + (int)threadIdx.x;
            if (p >= s.a && p < s.n - s.b && (i == 0 || k[u] >> above == prefix >> above))
                atomicAdd(&hist[k[u] >> shift & ((1 << digit_bits(i)) - 1)], 1);
        }
    }
    // rows that stay in any case, and those of the bar's weight, of every grain here
    __device__ __forceinline__ void grains(const EvictArgs &e, int n, int base, const Lot &s, uint32_t bar, int want) const {
        const int lane = threadIdx.x & 63, grain = evict_grain(e.row16);
        int *kept = e.kept + (size_t)n * e.grains, *ties = e.ties + (size_t)n * e.grains;
#pragma unroll
        for (int u = 0; u < KR; ++u) {
            const int p0 = base + u * ET + (int)(threadIdx.x & ~63u), p = p0 + lane;
            if (base + u * ET >= s.n) break;
            const bool in = p < s.n, mid = in && p >= s.a && p < s.n - s.b;
            const uint64_t more = __ballot(in && (!mid || (want > 0 && k[u] > bar)));
            const uint64_t same = __ballot(mid && want > 0 && k[u] == bar);
            // (a wave holds one grain or two)
            const int g = lane / grain;
            const uint64_t mask = grain == 64 ? ~0ull : 0xffffffffull << (32 * g);
            if (lane % grain == 0 && in) {
                kept[p0 / grain + g] = __popcll(more & mask);
                ties[p0 / grain + g] = __popcll(same & mask);
            }
        }
    }
};

// The largest digit with at least `want` rows at or above it, and `want` less the rows above it.
__device__ __forceinline__ int find_digit(const int *hist, int i, int &want, int (*waves)[2], int *pick) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    // thread t owns digits 2t and 2t + 1 from the top
    const int top = (1 << digit_bits(i)) - 1, d0 = top - 2 * tid, h0 = d0 >= 0 ? hist[d0] : 0, h1 = d0 >= 1 ? hist[d0 - 1] : 0;
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
    const int digit = pick[0];
    want -= pick[1];
    __syncthreads();
    return digit;
}

// From the grains' counts to the rows kept and the equal ones before each; of those the first `spare` stay.
__device__ __forceinline__ void sum_grains(const EvictArgs &e, int n, int num, int spare, int (*waves)[2]) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int *kept = e.kept + (size_t)n * e.grains, *ties = e.ties + (size_t)n * e.grains;
    int more0 = 0, same0 = 0;
    for (int g0 = 0; g0 < num; g0 += ET) {
        const int g = g0 + tid;
        const int m0 = g < num ? kept[g] : 0, t0 = g < num ? ties[g] : 0;
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
        if (g < num) {
            const int eq = same0 + t - t0; // equal ones before the grain
            ties[g] = eq;
            kept[g] = more0 + m - m0 + min(eq, spare);
        }
        more0 += mall;
        same0 += tall;
    }
}

__device__ __forceinline__ void clear(int *hist) {
    for (int i = threadIdx.x; i < EVICT_BINS; i += ET) hist[i] = 0;
    __syncthreads();
}

// One workgroup to a sequence.
template <int KR> __global__ __launch_bounds__(ET) void evict_choose_kernel(EvictArgs e) {
    __shared__ int hist[EVICT_BINS], waves[ET / 64][2], pick[2];
    const int n = blockIdx.x, tid = threadIdx.x, seg = evict_segment(e.row16);
    const Lot s = lot_of(e, n);
    const int nseg = (s.n + seg - 1) / seg, grain = evict_grain(e.row16);
    if (tid == 0) {
        e.lens_out[n] = s.k;
        e.ticket[n] = 0;
    }
    if (s.k == s.n) return; // (the move leaves such a sequence alone too)
    int *done = e.done + (size_t)n * e.segs;
    for (int i = tid; i < nseg; i += ET) done[i] = 0;
    Keys<KR> keys;
    keys.load(e, e.table + (size_t)n * e.cols, 0, s);
    int want = s.k - s.a - s.b; // rows that stay of those to choose among
    uint32_t bar = 0;
    if (want > 0)
        for (int i = 0; i < 3; ++i) {
            clear(hist);
            keys.count(hist, 0, s, bar, i);
            __syncthreads();
            bar |= (uint32_t)find_digit(hist, i, want, waves, pick) << digit_shift(i);
        }
    if (tid == 0) {
        e.bar[n] = bar;
        e.spare[n] = want;
    }
    keys.grains(e, n, 0, s, bar, want);
    __syncthreads();
    sum_grains(e, n, (s.n + grain - 1) / grain, want, waves);
}

// One of a sequence's chunks; pass 0 to 2 for the digits, 3 for the grains.
__global__ __launch_bounds__(ET) void evict_chunk_kernel(EvictArgs e, int pass) {
    constexpr int KR = EVICT_CHUNK / ET;
    __shared__ int hist[EVICT_BINS], waves[ET / 64][2], pick[2];
    const int n = blockIdx.x % e.N, chunk = blockIdx.x / e.N, base = chunk * EVICT_CHUNK, tid = threadIdx.x;
    const int seg = evict_segment(e.row16);
    const Lot s = lot_of(e, n);
    if (pass == 0 && chunk == 0 && tid == 0) {
        e.lens_out[n] = s.k;
        e.ticket[n] = 0;
        e.arrived[n] = 0;
    }
    if (s.k == s.n || base >= s.n) return;
    const int chunks = (s.n + EVICT_CHUNK - 1) / EVICT_CHUNK, nseg = (s.n + seg - 1) / seg, grain = evict_grain(e.row16);
    if (pass == 0) {
        int *done = e.done + (size_t)n * e.segs;
        for (int i = base / seg + tid; i < min(base / seg + EVICT_CHUNK / seg, nseg); i += ET) done[i] = 0;
    }
    Keys<KR> keys;
    keys.load(e, e.table + (size_t)n * e.cols, base, s);
    int want = s.k - s.a - s.b;
    uint32_t bar = 0;
    if (want > 0) {
        // the digit before: all chunks' histograms added up
        if (pass > 0) {
            if (pass > 1) {
                bar = e.state[(n * 3 + pass - 2) * 2];
                want = (int)e.state[(n * 3 + pass - 2) * 2 + 1];
            }
            const int *h = e.hist + ((size_t)((pass - 1) & 1) * e.N + n) * e.chunks * EVICT_BINS;
            for (int i = tid; i < EVICT_BINS; i += ET) {
                int x = 0;
#pragma unroll 8
                for (int c = 0; c < chunks; ++c) x += h[(size_t)c * EVICT_BINS + i];
                hist[i] = x;
            }
            __syncthreads();
            bar |= (uint32_t)find_digit(hist, pass - 1, want, waves, pick) << digit_shift(pass - 1);
            if (chunk == 0 && tid == 0) {
                e.state[(n * 3 + pass - 1) * 2] = bar;
                e.state[(n * 3 + pass - 1) * 2 + 1] = (uint32_t)want;
            }
        }
        if (pass < 3) {
            clear(hist);
            keys.count(hist, base, s, bar, pass);
            __syncthreads();
            int *h = e.hist + (((size_t)(pass & 1) * e.N + n) * e.chunks + chunk) * EVICT_BINS;
            for (int i = tid; i < EVICT_BINS; i += ET) h[i] = hist[i];
        }
    }
    if (pass < 3) return;
    if (chunk == 0 && tid == 0) {
        e.bar[n] = bar;
        e.spare[n] = want;
    }
    keys.grains(e, n, base, s, bar, want);
    // the last of the sequence's workgroups adds up what all have counted
    __syncthreads();
    if (tid == 0) pick[0] = __hip_atomic_fetch_add(&e.arrived[n], 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (pick[0] != chunks - 1) return;
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
    sum_grains(e, n, (s.n + grain - 1) / grain, want, waves);
}

// A segment of a sequence, as a workgroup's threads see it: each has a row of it, a wave a grain (or two
// waves' worth of threads have none).
struct Segment {
    int n, g, first, before, ties, spare, entry, slot;
    uint32_t bar;
    float weight;
    Lot s;
    // what the rows' choice hangs on, requested ...
    __device__ __forceinline__ void ask(const EvictArgs &e, int sequence, int ticket) {
        const int seg = evict_segment(e.row16), grain = evict_grain(e.row16), tid = threadIdx.x;
        n = sequence;
        g = ticket;
        s = lot_of(e, n);
        const size_t at = (size_t)n * e.grains;
        first = e.kept[at + g * seg / grain];
        const int mine = (g * seg + (row_in(e) ? (int)(tid & ~63u) : 0)) / grain;
        before = e.kept[at + mine];
        ties = e.ties[at + mine];
        bar = e.bar[n];
        spare = e.spare[n];
        entry = row_in(e) ? e.table[(size_t)n * e.cols + (unsigned)row(e) / (unsigned)e.page] : -1;
    }
    // ... and the row's weight
    __device__ __forceinline__ void look(const EvictArgs &e) {
        slot = slot_in(e, entry, row(e));
        weight = slot < 0 ? 0.f : e.weights[slot];
    }
    __device__ __forceinline__ int row(const EvictArgs &e) const { return g * evict_segment(e.row16) + (int)threadIdx.x; }
    __device__ __forceinline__ bool row_in(const EvictArgs &e) const {
        return (int)threadIdx.x < evict_segment(e.row16) && row(e) < s.n;
    }
};

__global__ __launch_bounds__(EM, 4) void evict_move_kernel(EvictArgs e) {
    __shared__ int from[EM], to[EM], counts[EM / 64], drawn[2];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row16 = e.row16, seg = evict_segment(row16);
    // as many tickets of a sequence are drawn as it has segments
    auto parts = [&](int i) { return move_segments(e, i, seg); };
    const Pieces all = Pieces::of(e.N, parts, lane);
    int b = blockIdx.x;
    if (b >= all.total) return;
    // A segment's ticket is drawn, and what its rows' choice hangs on requested, while the one before it is moved.
    Segment c, next;
    {
        int n, any;
        all.find(parts, b, lane, n, any);
        if (tid == 0) drawn[0] = atomicAdd(&e.ticket[n], 1);
        __syncthreads();
        c.ask(e, n, __builtin_amdgcn_readfirstlane(drawn[0]));
        c.look(e);
    }
    for (int turn = 1;; turn ^= 1) {
        b += gridDim.x;
        const bool more = b < all.total;
        int n2 = 0, any;
        if (more) {
            all.find(parts, b, lane, n2, any);
            if (tid == 0) drawn[turn] = atomicAdd(&e.ticket[n2], 1);
        }
        // which rows stay, and where they go
        const Lot &s = c.s;
        const int *tb = e.table + (size_t)c.n * e.cols;
        int *done = e.done + (size_t)c.n * e.segs;
        const int p = c.row(e), first = c.first, g = c.g;
        const uint32_t key = c.slot < 0 ? 0u : key_of(c.weight);
        const bool in = c.row_in(e), mid = in && p >= s.a && p < s.n - s.b, tie = mid && c.spare > 0 && key == c.bar;
        const uint64_t below = (1ull << lane) - 1, eq = __ballot(tie);
        const bool stay = in && (!mid || (c.spare > 0 && key > c.bar) || (tie && c.ties + __popcll(eq & below) < c.spare));
        const uint64_t st = __ballot(stay);
        const int rank = c.before - first + __popcll(st & below); // among the segment's
        int dst = -1;
        if (stay) {
            dst = slot_in(e, tb[(unsigned)(first + rank) / (unsigned)e.page], first + rank);
            from[rank] = c.slot;
            to[rank] = dst;
        }
        if (lane == 0) counts[wave] = __popcll(st);
        __syncthreads();
        const int count = (counts[0] + counts[1]) + (counts[2] + counts[3]), pieces = count * row16;
        // the rows, into registers (a segment whose rows all stay where they are has nothing to read)
        const bool moves = count > 0 && first < g * seg + min(seg, s.n - g * seg) - count;
        u32x4 x[EV];
        u32x4 *pool = (u32x4 *)e.cache;
        if (moves) {
#pragma unroll
            for (int v = 0; v < EV; ++v) {
                if (v * EM >= pieces) continue;
                const int i = min(tid + v * EM, pieces - 1), row = (unsigned)i / (unsigned)row16, src = from[row];
                x[v] = load16(src < 0 ? (const void *)&mla_zeros
                                      : (const void *)(pool + (size_t)(unsigned)src * row16 + (i - row * row16)));
            }
        }
        if (more) next.ask(e, n2, __builtin_amdgcn_readfirstlane(drawn[turn]));
        // All of it is here before the flag says so. (What the flag orders are these reads, done by now, and others'
        // writes: it has nothing to publish, so it needs no release, which would write back the L2.)
        wait_vmem();
        __syncthreads();
        if (tid == 0) __hip_atomic_store(&done[g], 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (more) next.look(e);
        if (moves) {
            // the rows' new places hold rows of at most two segments before this one
            if (tid == 0) {
                const int g0 = first / seg, g1 = min((first + count - 1) / seg, g - 1);
                for (int i = g0; i <= g1; ++i)
                    while (!__hip_atomic_load(&done[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) __builtin_amdgcn_s_sleep(2);
            }
            __syncthreads();
#pragma unroll
            for (int v = 0; v < EV; ++v) {
                if (v * EM >= pieces) continue;
                const int i = tid + v * EM, row = (unsigned)min(i, pieces - 1) / (unsigned)row16;
                if (i < pieces && from[row] >= 0 && to[row] >= 0)
                    pool[(size_t)(unsigned)to[row] * row16 + (i - row * row16)] = x[v];
            }
            if (stay && c.slot >= 0 && dst >= 0) e.weights[dst] = c.weight;
        }
        if (!more) break;
        __syncthreads(); // (from and to are read)
        c = next;
    }
}

hipError_t launch_evict_choose(const EvictArgs &a, hipStream_t st) {
    if (a.chunks == 1) {
        if ((long long)a.cols * a.page <= 8 * ET) hipLaunchKernelGGL(evict_choose_kernel<8>, dim3(a.N), dim3(ET), 0, st, a);
        else hipLaunchKernelGGL(evict_choose_kernel<EVICT_ONE / ET>, dim3(a.N), dim3(ET), 0, st, a);
        return hipGetLastError();
    }
    for (int pass = 0; pass < 4; ++pass) {
        hipLaunchKernelGGL(evict_chunk_kernel, dim3((unsigned)((long long)a.N * a.chunks)), dim3(ET), 0, st, a, pass);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}
hipError_t launch_evict_move(const EvictArgs &a, hipStream_t st) {
    // as many workgroups as the chip holds (four to a CU); how many segments there are is known on the GPU alone
    const long long most = (long long)a.N * a.segs, held = 4 * MLA_CUS;
    hipLaunchKernelGGL(evict_move_kernel, dim3((unsigned)(most < held ? most : held)), dim3(EM), 0, st, a);
    return hipGetLastError();
}

} // namespace gdn
