// nmpages.hip -- nm_kv_plan: the book of a cache's pages, kept on the GPU.
//
// All of a step's decisions are sums over the sequences in order (pages given back,
// pages and rows asked for), so one block makes them: thread t has the sequences
// t c .. t c + c - 1, adds up its own, and a scan over the block's 1024 threads says
// where each begins.  Pages and rows are then dealt with one a thread, each finding
// its sequence by a binary search in the scanned sums, so that one sequence of many
// pages costs no more than many of one.
//   The rows (slots, positions, new entries of the table) follow in the same block
// while there are few, else in a launch of their own over the whole GPU; what they
// need of the decisions is in `scratch` by then.
// Latency bounds it: the decisions are a chain of a few loads, two scans and a
// search, the rows move 12 bytes each.

#include <hip/hip_runtime.h>

#include <cstdint>

#include "nm_device.h"
#include "nm_serve.h"

namespace {

using namespace nmd;

constexpr int kThreads = nms::kPlanThreads;

struct PlanArgs {
    int32_t* table;
    int32_t* lens;
    int32_t* free;
    int32_t* n_free;
    int32_t* first_pop;             // [B] scratch: pages taken off the stack before b's; [B]: pages on it before the first
    const int32_t* adds;
    int32_t* starts;
    int64_t* slots;
    int32_t* positions;
    int32_t* granted;
    int B, width, n_pages, shift;   // page_size = 1 << shift
    int rows;
    int each;                       // sequences of a thread
};

__device__ __forceinline__ int64_t pages_of(int64_t tokens, int shift) { return (tokens + (1 << shift) - 1) >> shift; }

// What one sequence asks for.
struct Request {
    int len, held;          // tokens (0 of a padding row) and pages now
    int drop, freed;        // tokens and pages given back
    int grow, want;         // tokens and pages asked for; 0 where the table's row is too short
    bool live;
};

__device__ __forceinline__ Request request(const PlanArgs& A, int b)
{
    const int len = A.lens[b];
    const int64_t add = A.adds[b];
    Request q;
    q.live = len >= 0;
    q.len = max(len, 0);
    // a length above what the row holds has no further pages
    q.held = (int)min(pages_of(q.len, A.shift), (int64_t)A.width);
    q.drop = q.live && add < 0 ? (int)min(-add, (int64_t)q.len) : 0;
    q.freed = q.held - (int)min(pages_of(q.len - q.drop, A.shift), (int64_t)A.width);
    const int64_t to = q.len + add, need = pages_of(to, A.shift);
    const bool fits = q.live && add > 0 && to <= INT32_MAX && need <= A.width;
    q.grow = fits ? (int)add : 0;
    q.want = fits ? (int)need - q.held : 0;
    return q;
}

// Inclusive sums over the block's threads, in `sums`; returns the total.
__device__ __forceinline__ int64_t scan(int64_t x, int64_t* sums, int64_t* waves)
{
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
#pragma unroll
    for (int i = 1; i < 64; i *= 2) {
        const int64_t y = __shfl_up(x, i);
        x += lane >= i ? y : 0;
    }
    if (lane == 63)
        waves[wave] = x;
    __syncthreads();
    int64_t before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
        before += w < wave ? waves[w] : 0;
        total += waves[w];
    }
    sums[threadIdx.x] = x + before;
    __syncthreads();
    return total;
}

// The first of n entries that is above x (n - 1 if none is).
template <class T>
__device__ __forceinline__ int above(const T* sums, int n, int64_t x)
{
    int lo = 0;
    for (int step = n; step > 0;) {
        const int half = step / 2;
        if (lo + half < n && sums[lo + half] <= x) {
            lo += half + 1;
            step -= half + 1;
        } else {
            step = half;
        }
    }
    return min(lo, n - 1);
}

// Row r is token `at` of sequence b, which held `len` tokens on `held` pages.
__device__ __forceinline__ void row(const PlanArgs& A, int r, int b, int at, int held, int first_pop, int room)
{
    const int index = at >> A.shift, place = at & ((1 << A.shift) - 1);
    int32_t* entry = A.table + (int64_t)b * A.width + index;
    int page;
    if (index < held) {
        page = *entry;
    } else {
        page = A.free[room - 1 - (first_pop + index - held)];
        if (place == 0)
            *entry = page;
    }
    A.slots[r] = page < 0 ? -1 : ((int64_t)page << A.shift) + place;
    A.positions[r] = at;
}

__device__ __forceinline__ void no_row(const PlanArgs& A, int r)
{
    A.slots[r] = -1;
    A.positions[r] = 0;
}

__global__ __launch_bounds__(kThreads) void plan_kernel(const PlanArgs A, int with_rows)
{
    __shared__ int64_t sums[kThreads], pops[kThreads], waves[kThreads / 64];
    __shared__ int held_of[kThreads], len_of[kThreads];
    __shared__ int64_t stop_rows, stop_pages;
    __shared__ int stop;
    const int tid = threadIdx.x, b0 = min(tid * A.each, A.B), b1 = min(b0 + A.each, A.B);
    if (tid == 0)
        stop = A.B;
    const int n_free = min(max(A.n_free[0], 0), A.n_pages);

    // Pages that come back, the first one on top.
    int64_t own = 0;
    for (int b = b0; b < b1; ++b)
        own += request(A, b).freed;
    const int64_t freed = scan(own, sums, waves);
    for (int64_t k = tid; k < freed; k += kThreads) {
        const int t = above(sums, kThreads, k);
        int64_t in = k - (t > 0 ? sums[t - 1] : 0);
        int b = t * A.each;
        Request q = request(A, b);
        while (in >= q.freed) {
            in -= q.freed;
            q = request(A, ++b);
        }
        const int64_t to = n_free + freed - 1 - k;
        if (to < A.n_pages)
            A.free[to] = A.table[(int64_t)b * A.width + q.held - q.freed + in];
    }
    const int64_t room = min(n_free + freed, (int64_t)A.n_pages);

    // What is asked for, in order, until pages or rows run out.
    int64_t want = 0, grow = 0;
    for (int b = b0; b < b1; ++b) {
        const Request q = request(A, b);
        want += q.want;
        grow += q.grow;
    }
    __syncthreads();
    const int64_t all_pages = scan(want, pops, waves);
    __syncthreads();
    const int64_t all_rows = scan(grow, sums, waves);
    const int64_t pages0 = pops[tid] - want, rows0 = sums[tid] - grow;
    if (pops[tid] > room || sums[tid] > A.rows) {
        int64_t p = pages0, n = rows0;
        for (int b = b0; b < b1; ++b) {
            const Request q = request(A, b);
            if (p + q.want > room || n + q.grow > A.rows) {
                atomicMin(&stop, b);
                break;
            }
            p += q.want;
            n += q.grow;
        }
    }
    __syncthreads();
    const int last = stop;
    if (last < A.B && b0 <= last && last < b1) {
        int64_t p = pages0, n = rows0;
        for (int b = b0; b < last; ++b) {
            const Request q = request(A, b);
            p += q.want;
            n += q.grow;
        }
        stop_pages = p;
        stop_rows = n;
    }
    __syncthreads();
    const int64_t got_rows = last < A.B ? stop_rows : all_rows, got_pages = last < A.B ? stop_pages : all_pages;
    {
        int64_t p = pages0, n = rows0;
        for (int b = b0; b < b1; ++b) {
            const Request q = request(A, b);
            const bool ok = b < last;
            const int change = (ok ? q.grow : 0) - q.drop;
            if (with_rows) {                    // one sequence a thread
                held_of[tid] = q.held;
                len_of[tid] = q.len;
            }
            A.first_pop[b] = (int)min(p, room);
            p += q.want;
            n += q.grow;
            A.granted[b] = change;
            A.starts[b + 1] = (int)(ok ? n : got_rows);
            if (change != 0)
                A.lens[b] = q.len + change;
        }
    }
    if (tid == 0) {
        A.starts[0] = 0;
        A.first_pop[A.B] = (int)room;
        A.n_free[0] = (int)(room - got_pages);
    }
    if (!with_rows)
        return;
    __syncthreads();
    for (int r = tid; r < A.rows; r += kThreads) {
        if (r >= got_rows) {
            no_row(A, r);
            continue;
        }
        const int b = above(sums, A.B, r);
        row(A, r, b, len_of[b] + r - (int)(b > 0 ? sums[b - 1] : 0), held_of[b], (int)(b > 0 ? pops[b - 1] : 0), (int)room);
    }
}

// The rows alone, kRowsBlock a block.  A block finds the sequences of its first and last
// row, 64 at a time, and its threads search between them.
constexpr int kRowsBlock = 256;

__device__ __forceinline__ int sequence_of(const int32_t* ends, int n, int r, int lane)
{
    int lo = 0;                                     // the first end above r
    while (n > 1) {
        const int step = (n + 63) / 64, at = min((lane + 1) * step, n) - 1;
        const int below = __popcll(__ballot(lane * step < n && ends[lo + at] <= r));
        const int skip = min(below * step, n - 1);
        lo += skip;
        n = min(step, n - skip);
    }
    return lo;
}

__global__ __launch_bounds__(kRowsBlock) void rows_kernel(const PlanArgs A)
{
    const int lane = threadIdx.x % 64;
    const int64_t r0 = (int64_t)flat_block() * kRowsBlock, r = r0 + threadIdx.x;
    if (r0 >= A.rows)
        return;
    const int n = A.starts[A.B], room = A.first_pop[A.B];
    if (r0 < n) {
        const int32_t* ends = A.starts + 1;
        const int first = sequence_of(ends, A.B, (int)r0, lane);
        const int last = sequence_of(ends, A.B, (int)min(r0 + kRowsBlock, (int64_t)n) - 1, lane);
        if (r < n) {
            const int b = first + above(ends + first, last - first + 1, r);
            const int len = A.lens[b] - A.granted[b];
            row(A, (int)r, b, len + (int)r - A.starts[b], (int)pages_of(len, A.shift), A.first_pop[b], room);
            return;
        }
    }
    if (r < A.rows)
        no_row(A, (int)r);
}

}  // namespace

int nmk::kv_plan(const nm_kv_pages& p, const int32_t* adds, int64_t rows, int32_t* starts, int64_t* slots,
                 int32_t* positions, int32_t* granted, void* stream)
{
    PlanArgs A;
    A.table = p.table;
    A.lens = p.lens;
    A.free = p.free;
    A.n_free = p.n_free;
    A.first_pop = static_cast<int32_t*>(p.scratch);
    A.adds = adds;
    A.starts = starts;
    A.slots = slots;
    A.positions = positions;
    A.granted = granted;
    A.B = (int)p.B;
    A.width = (int)p.width;
    A.n_pages = (int)p.n_pages;
    A.shift = __builtin_ctz((unsigned)p.page_size);
    A.rows = (int)rows;
    A.each = (int)nma::ceil_div(p.B, kThreads);
    hipStream_t s = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    const bool with_rows = A.each == 1 && rows <= nms::kPlanRows;
    hipLaunchKernelGGL(plan_kernel, dim3(1), dim3(kThreads), 0, s, A, with_rows ? 1 : 0);
    if (!with_rows && rows > 0)
        hipLaunchKernelGGL(rows_kernel, flat_grid(nma::ceil_div(rows, kRowsBlock)), dim3(kRowsBlock), 0, s, A);
    return hipGetLastError() == hipSuccess ? NM_OK : NM_ERR_HIP;
}
