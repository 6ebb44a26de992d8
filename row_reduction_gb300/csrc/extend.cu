// extend.cu -- the pages, slots and positions of a step's tokens.
//
//   n_s = ceil((lengths + counts) / page) - ceil(lengths / page),
//   e_s = n_0 + .. + n_(s-1)
//
// Up to kOne sequences take one kernel: every CTA adds up all of them for
// itself (two prefix sums, tokens and pages, kept in shared memory; the counts
// come from L2) and then has its share of the new pages and of the rows, each
// of which finds its sequence by halving.  A row in a new page takes it from the
// list, as the CTA that writes the table does, so that no CTA waits for
// another.  More sequences take two kernels: one CTA goes through them in order
// and gives out the pages, then a thread per row.
//
// Bound: latency.  256 sequences of a token each 4.3 us, 1024 6.5 (sums that every
// CTA makes for itself, 64-bit divisions by the page size among them), 1024 with
// 107 thousand rows 10 (two kernels: 8.0 and 12.9): a row is a thread's one search,
// two divisions and a page.  4096 with a token each 17 us; by two kernels 4097 24,
// 65536 232, where one CTA goes through the sequences.
#include "mt_decoder.cuh"

namespace mt {
namespace {

constexpr int kScan = 1024;
constexpr int kRowThreads = 256;
constexpr int64_t kMost = INT32_MAX;

// What a sequence holds and asks for.
struct Asked {
    int64_t length, count;  // tokens
    int64_t held, need;     // pages; need is 0 where they do not fit
    bool fits;
};
__device__ __forceinline__ Asked asked(const mt_cache_extend_call_t &c,
                                       int64_t s) {
    Asked a;
    a.length = max(c.lengths[s], 0);
    a.count = max(c.counts[s], 0);
    a.held = (a.length + c.page_size - 1) / c.page_size;
    const int64_t want = (a.length + a.count + c.page_size - 1) / c.page_size;
    a.fits = a.length + a.count <= kMost && (want == a.held || want <= c.pages);
    a.need = a.fits ? want - a.held : 0;
    return a;
}

// Exclusive sums over the CTA, and their totals.
struct Pair {
    int64_t tokens, pages;
};
__device__ __forceinline__ Pair scan(Pair v, Pair &total) {
    __shared__ Pair warps[kScan / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Pair in = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(kFull, in.tokens, o);
        const int64_t p = __shfl_up_sync(kFull, in.pages, o);
        if (lane >= o) {
            in.tokens += t;
            in.pages += p;
        }
    }
    __syncthreads();  // warps[] of the call before
    if (lane == 31) warps[warp] = in;
    __syncthreads();
    Pair before = {0, 0};
    total = {0, 0};
    for (int w = 0; w < (int)blockDim.x >> 5; ++w) {
        if (w == warp) before = total;
        total.tokens += warps[w].tokens;
        total.pages += warps[w].pages;
    }
    return {before.tokens + in.tokens - v.tokens,
            before.pages + in.pages - v.pages};
}

__global__ void __launch_bounds__(kScan)
    extend_kernel(const mt_cache_extend_call_t c) {
    grid_launch_dependents();
    grid_wait_prerequisites();
    const int64_t free_pages = min(max(*c.free_count, 0), c.free_size);
    Pair carry = {0, 0};
    int64_t used = 0;
    for (int64_t s0 = 0; s0 < c.sequences; s0 += blockDim.x) {
        const int64_t s = s0 + threadIdx.x;
        const bool in = s < c.sequences;
        Asked a = {};
        if (in) a = asked(c, s);
        Pair total;
        Pair at = scan({a.count, a.need}, total);
        at.tokens += carry.tokens;
        at.pages += carry.pages;
        if (in) {
            const bool served =
                a.fits && (a.need == 0 || at.pages + a.need <= free_pages);
            c.offsets[s] = (int32_t)min(at.tokens, kMost);
            c.new_lengths[s] = (int32_t)(a.length + (served ? a.count : 0));
            if (served && a.need > 0) {
                used = at.pages + a.need;
                int32_t *row = c.table + s * c.table_stride + a.held;
                const int32_t *from =
                    c.free_pages + (free_pages - 1 - at.pages);
                for (int64_t i = 0; i < a.need; ++i) row[i] = from[-i];
            }
        }
        carry.tokens += total.tokens;
        carry.pages += total.pages;
    }
    // The last served sequence that took pages has the largest sum.
    __shared__ unsigned long long most;
    __syncthreads();
    if (threadIdx.x == 0) most = 0;
    __syncthreads();
    if (used > 0) atomicMax(&most, (unsigned long long)used);
    __syncthreads();
    if (threadIdx.x == 0) {
        c.offsets[c.sequences] = (int32_t)min(carry.tokens, kMost);
        *c.new_free_count = (int32_t)(free_pages - (int64_t)most);
    }
}

__global__ void __launch_bounds__(kRowThreads)
    extend_rows_kernel(const mt_cache_extend_call_t c) {
    grid_launch_dependents();
    grid_wait_prerequisites();
    const int64_t r = (int64_t)blockIdx.x * kRowThreads + threadIdx.x;
    if (r >= c.rows) return;
    int64_t slot = -1;
    int32_t place = 0;
    if (c.sequences > 0 && r < c.offsets[c.sequences]) {
        int lo = 0, hi = c.sequences;  // offsets[lo] <= r < offsets[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (c.offsets[mid] <= r) lo = mid; else hi = mid;
        }
        const Asked a = asked(c, lo);
        const int64_t p = a.length + (r - c.offsets[lo]);
        place = (int32_t)min(p, kMost);
        if (c.new_lengths[lo] - a.length == a.count && p / c.page_size < c.pages) {
            const int32_t id = c.table[lo * c.table_stride + p / c.page_size];
            if (id >= 0) slot = (int64_t)id * c.page_size + p % c.page_size;
        }
    }
    c.slots[r] = slot;
    c.positions[r] = place;
}

// The last place of an ascending array (n + 1 values) whose value is at most
// v < at[n].
__device__ __forceinline__ int place_in(const int32_t *at, int n, int64_t v) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (at[mid] <= v) lo = mid; else hi = mid;
    }
    return lo;
}

constexpr int kOne = 4096;          // sequences of the one kernel
constexpr int kOneThreads = 256;
__global__ void __launch_bounds__(kOneThreads)
    extend_one_kernel(const mt_cache_extend_call_t c) {
    extern __shared__ int32_t sums[];
    int32_t *offsets = sums, *pages = sums + c.sequences + 1;
    __shared__ int32_t most[kOneThreads / 32];
    grid_launch_dependents();
    grid_wait_prerequisites();
    const int n = c.sequences, tid = threadIdx.x;
    const int32_t held_free = min(max(*c.free_count, 0), c.free_size);
    // A run of sequences per thread; the sums stop at the type's largest.
    const int each = (n + kOneThreads - 1) / kOneThreads;
    const int s0 = min(tid * each, n), s1 = min(s0 + each, n);
    Pair mine = {0, 0};
    for (int s = s0; s < s1; ++s) {
        const Asked a = asked(c, s);
        mine.tokens += a.count;
        mine.pages += a.need;
    }
    Pair total;
    Pair at = scan(mine, total);
    int32_t used = 0;  // pages of the list that are given out
    for (int s = s0; s < s1; ++s) {
        const Asked a = asked(c, s);
        const bool served =
            a.fits && (a.need == 0 || at.pages + a.need <= held_free);
        offsets[s] = (int32_t)min(at.tokens, kMost);
        pages[s] = (int32_t)min(at.pages, kMost);
        if (served && a.need > 0) used = (int32_t)(at.pages + a.need);
        if (s % (int)gridDim.x == (int)blockIdx.x) {
            c.offsets[s] = offsets[s];
            c.new_lengths[s] = (int32_t)(a.length + (served ? a.count : 0));
        }
        at.tokens += a.count;
        at.pages += a.need;
    }
    used = __reduce_max_sync(kFull, used);
    if ((tid & 31) == 0) most[tid >> 5] = used;
    if (tid == 0) {
        offsets[n] = (int32_t)min(total.tokens, kMost);
        pages[n] = (int32_t)min(total.pages, kMost);
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kOneThreads / 32; ++x) used = max(used, most[x]);
    if (tid == 0 && blockIdx.x == 0) {
        c.offsets[n] = offsets[n];
        *c.new_free_count = held_free - used;
    }
    const int64_t step = (int64_t)gridDim.x * kOneThreads;
    const int64_t first = (int64_t)blockIdx.x * kOneThreads + tid;
    for (int64_t i = first; i < used; i += step) {
        const int s = place_in(pages, n, i);
        c.table[s * c.table_stride + asked(c, s).held + (i - pages[s])] =
            c.free_pages[held_free - 1 - i];
    }
    for (int64_t r = first; r < c.rows; r += step) {
        int64_t slot = -1;
        int32_t place = 0;
        if (n > 0 && r < offsets[n]) {
            const int s = place_in(offsets, n, r);
            const Asked a = asked(c, s);
            const int64_t p = a.length + (r - offsets[s]);
            const int64_t page = p / c.page_size;
            place = (int32_t)min(p, kMost);
            if (a.fits && page < c.pages &&
                (a.need == 0 || pages[s] + a.need <= held_free)) {
                const int32_t id =
                    page < a.held
                        ? c.table[s * c.table_stride + page]
                        : c.free_pages[held_free - 1 - pages[s] -
                                       (page - a.held)];
                if (id >= 0)
                    slot = (int64_t)id * c.page_size + (p - page * c.page_size);
            }
        }
        c.slots[r] = slot;
        c.positions[r] = place;
    }
}

}  // namespace

cudaError_t launch_cache_extend(const mt_cache_extend_call_t &c,
                                cudaStream_t s) {
    if (c.sequences <= kOne) {
        int sms = 0;
        const cudaError_t e = current_sm_count(&sms);
        if (e != cudaSuccess) return e;
        // a thread for each row, up to four CTAs on an SM
        int64_t grid = (c.rows + kOneThreads - 1) / kOneThreads;
        if (grid < c.sequences / 32) grid = c.sequences / 32;
        if (grid > 4LL * sms) grid = 4LL * sms;
        if (grid < 1) grid = 1;
        return launch_dependent(extend_one_kernel, grid, kOneThreads,
                                (size_t)2 * (c.sequences + 1) *
                                    sizeof(int32_t), s, c);
    }
    cudaError_t e = launch_dependent(extend_kernel, 1, kScan, 0, s, c);
    if (e == cudaSuccess && c.rows > 0)
        e = launch_dependent(extend_rows_kernel,
                             (c.rows + kRowThreads - 1) / kRowThreads,
                             kRowThreads, 0, s, c);
    return e;
}

}  // namespace mt
