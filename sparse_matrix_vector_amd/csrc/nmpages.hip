// nmpages.hip -- nm_kv_plan: the book of a cache's pages, kept on the GPU.
//
// All of a step's decisions are sums over the sequences in order (pages given back,
// pages and rows asked for), so one block makes them: thread t has the sequences
// t c .. t c + c - 1, adds up its own, and a scan over the block's threads says
// where each begins.  Pages and rows are then dealt out to the threads, each finding
// its sequence by a binary search in the scanned sums, so that one sequence of many
// pages costs no more than many of one (48 sequences that end, 2900 pages: 7.5 us).
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

__device__ __forceinline__ Request request(const PlanArgs& A, int len, int64_t add)
{
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

__device__ __forceinline__ Request request(const PlanArgs& A, int b) { return request(A, A.lens[b], A.adds[b]); }

// Four int32 of a thread, at any 4-byte aligned address.
typedef int i32x4 __attribute__((ext_vector_type(4), aligned(4)));

// What sequences give back and ask for, added up: pages (below 2^31, as B * width is) and rows,
// of which more than `most` = rows + 1 count as that many (they do not fit whatever follows).
struct Sums {
    uint32_t freed, want, grow;
};

__device__ __forceinline__ Sums plus(Sums a, Sums b, uint32_t most)
{
    const uint64_t grow = (uint64_t)a.grow + b.grow;
    return {a.freed + b.freed, a.want + b.want, grow > most ? most : (uint32_t)grow};
}

// Inclusive sums over the lanes of a wave, of which the first N count.
template <int N>
__device__ __forceinline__ Sums scan_wave(Sums x, uint32_t most, int lane)
{
#pragma unroll
    for (int i = 1; i < N; i *= 2) {
        const Sums y = {__shfl_up(x.freed, i), __shfl_up(x.want, i), __shfl_up(x.grow, i)};
        if (lane >= i)
            x = plus(x, y, most);
    }
    return x;
}

// Inclusive sums over the block's threads, in sums[1 ..] with nothing in sums[0]; returns the totals.
template <int NT>
__device__ __forceinline__ Sums scan(Sums x, uint32_t most, Sums* sums, Sums* waves)
{
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    x = scan_wave<64>(x, most, lane);
    if (threadIdx.x == 0)
        sums[0] = Sums{0, 0, 0};
    if constexpr (NT > 64) {
        if (lane == 63)
            waves[wave] = x;
        __syncthreads();
        // every wave adds up the waves' totals for itself
        const Sums y = scan_wave<NT / 64>(lane < NT / 64 ? waves[lane] : Sums{0, 0, 0}, most, lane);
        if (wave > 0)
            x = plus(x, {__shfl(y.freed, wave - 1), __shfl(y.want, wave - 1), __shfl(y.grow, wave - 1)}, most);
    }
    sums[1 + threadIdx.x] = x;
    __syncthreads();
    return sums[NT];
}

// The first of n entries whose value is above x (n - 1 if none is).
template <class F>
__device__ __forceinline__ int above(F value, int n, int64_t x)
{
    int lo = 0;
    for (int left = n - 1; left > 0;) {                 // among lo .. lo + left
        const int half = left / 2;
        if (value(lo + half) <= x) {
            lo += half + 1;
            left -= half + 1;
        } else {
            left = half;
        }
    }
    return lo;
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

// NT threads with EACH sequences, kept in registers; EACH 0: any number of sequences, read again
// whenever they are looked at.
template <int NT, int EACH>
__global__ __launch_bounds__(NT) void plan_kernel(const PlanArgs A, int with_rows)
{
    __shared__ Sums sums[NT + 1], waves[NT / 64];
    __shared__ int held_of[EACH == 1 ? NT : 1], len_of[EACH == 1 ? NT : 1], kept_of[EACH == 1 ? NT : 1];
    __shared__ int stop;
    __shared__ uint32_t stop_rows, stop_pages;
    constexpr int kKept = EACH ? EACH : 1;
    const int each = EACH ? EACH : A.each;
    const int tid = threadIdx.x, b0 = min(tid * each, A.B), b1 = min(b0 + each, A.B);
    const int n_free = min(max(A.n_free[0], 0), A.n_pages);
    if (tid == 0)
        stop = A.B;
    Request kept[kKept];
    const uint32_t most = (uint32_t)A.rows + 1;
    Sums own = {0, 0, 0};
    const auto asked = [&](const Request& q) { return Sums{(uint32_t)q.freed, (uint32_t)q.want, (uint32_t)q.grow}; };
    const auto count = [&](const Request& q) { own = plus(own, asked(q), most); };
    int32_t first[kKept];               // the first page that each gives back
    i32x4 lens = {-1, -1, -1, -1}, adds = {0, 0, 0, 0};
    if constexpr (EACH > 0) {
        if (EACH == 4 && b0 + 4 <= b1) {
            lens = *reinterpret_cast<const i32x4*>(A.lens + b0);
            adds = *reinterpret_cast<const i32x4*>(A.adds + b0);
        } else {
#pragma unroll
            for (int i = 0; i < EACH; ++i)
                if (b0 + i < b1) {
                    lens[i] = A.lens[b0 + i];
                    adds[i] = A.adds[b0 + i];
                }
        }
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            kept[i] = request(A, (int)lens[i], (int)adds[i]);       // a padding row behind the last
            first[i] = kept[i].freed > 0 ? A.table[(int64_t)(b0 + i) * A.width + kept[i].held - kept[i].freed] : 0;
            count(kept[i]);
        }
    } else {
        for (int b = b0; b < b1; ++b)
            count(request(A, b));
    }
    // f(b, its request) for the thread's sequences, in order
    const auto walk = [&](auto f) {
        if constexpr (EACH > 0) {
#pragma unroll
            for (int i = 0; i < EACH; ++i)
                if (b0 + i < b1)
                    f(b0 + i, kept[i]);
        } else {
            for (int b = b0; b < b1; ++b)
                f(b, request(A, b));
        }
    };
    const Sums all = scan<NT>(own, most, sums, waves), before = sums[tid];

    // Pages that come back, the first one on top: by their own threads where those have few each, else
    // one a thread in turn.
    const int64_t top = (int64_t)n_free + all.freed - 1;
    const auto give = [&](int64_t k, int b, const Request& q, int64_t in) {
        if (top - k < A.n_pages)
            A.free[top - k] = A.table[(int64_t)b * A.width + q.held - q.freed + in];
    };
    if (all.freed > 0) {
        if (__syncthreads_and(own.freed <= 8)) {
            int64_t k = before.freed;
            walk([&](int b, const Request& q) {
                for (int in = 0; in < q.freed; ++in, ++k) {
                    if (EACH > 0 && in == 0) {
                        if (top - k < A.n_pages)
                            A.free[top - k] = first[EACH > 0 ? b - b0 : 0];
                    } else {
                        give(k, b, q, in);
                    }
                }
            });
        } else if constexpr (EACH == 1) {
            // eight in a row a thread, one search for all and no load behind another
            constexpr int kRun = 8;
            kept_of[tid] = kept[0].held - kept[0].freed;
            __syncthreads();
            for (int64_t k0 = (int64_t)tid * kRun; k0 < all.freed; k0 += kRun * NT) {
                int32_t page[kRun];
                int b = above([&](int t) { return sums[t + 1].freed; }, NT, k0);
#pragma unroll
                for (int i = 0; i < kRun; ++i) {
                    const int64_t k = min(k0 + i, (int64_t)all.freed - 1);
                    while (sums[b + 1].freed <= k)
                        ++b;
                    page[i] = A.table[(int64_t)b * A.width + kept_of[b] + (k - sums[b].freed)];
                }
#pragma unroll
                for (int i = 0; i < kRun; ++i)
                    if (k0 + i < all.freed && top - k0 - i < A.n_pages)
                        A.free[top - k0 - i] = page[i];
            }
        } else {
            for (int64_t k = tid; k < all.freed; k += NT) {
                const int t = above([&](int i) { return sums[i + 1].freed; }, NT, k);
                int64_t in = k - sums[t].freed;
                int b = t * each;
                Request q = request(A, b);
                while (in >= q.freed) {
                    in -= q.freed;
                    q = request(A, ++b);
                }
                give(k, b, q, in);
            }
            __syncthreads();                        // others' lens are read here
        }
    }
    const uint32_t room = (uint32_t)min(top + 1, (int64_t)A.n_pages);

    // What is asked for, in order, until pages or rows run out: at sequence `last`, if at all.
    int last = A.B;
    uint32_t got_rows = all.grow, got_pages = all.want;
    if (all.want > room || all.grow == most) {          // the same for all threads
        if (sums[tid + 1].want > room || sums[tid + 1].grow == most) {
            Sums x = before;
            int first = A.B;
            walk([&](int b, const Request& q) {
                x = plus(x, asked(q), most);
                if (first == A.B && (x.want > room || x.grow == most))
                    first = b;
            });
            atomicMin(&stop, first);
        }
        __syncthreads();
        last = stop;
        if (b0 <= last && last < b1) {
            Sums x = before;
            walk([&](int b, const Request& q) {
                if (b < last)
                    x = plus(x, asked(q), most);
            });
            stop_pages = x.want;
            stop_rows = x.grow;
        }
        __syncthreads();
        got_rows = stop_rows;
        got_pages = stop_pages;
    }
    if constexpr (EACH == 4) {
        Sums x = before;
        i32x4 pops, granted, ends;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Request& q = kept[i];
            const bool ok = b0 + i < last;
            granted[i] = (ok ? q.grow : 0) - q.drop;
            lens[i] = granted[i] != 0 ? q.len + granted[i] : lens[i];
            pops[i] = (int)min(x.want, room);
            x = plus(x, asked(q), most);
            ends[i] = (int)(ok ? x.grow : got_rows);
        }
        if (b0 + 4 <= b1) {
            *reinterpret_cast<i32x4*>(A.first_pop + b0) = pops;
            *reinterpret_cast<i32x4*>(A.granted + b0) = granted;
            *reinterpret_cast<i32x4*>(A.starts + b0 + 1) = ends;
            *reinterpret_cast<i32x4*>(A.lens + b0) = lens;
        } else {
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (b0 + i < b1) {
                    A.first_pop[b0 + i] = pops[i];
                    A.granted[b0 + i] = granted[i];
                    A.starts[b0 + i + 1] = ends[i];
                    A.lens[b0 + i] = lens[i];
                }
        }
    } else {
        Sums x = before;
        walk([&](int b, const Request& q) {
            const bool ok = b < last;
            const int change = (ok ? q.grow : 0) - q.drop;
            if constexpr (EACH == 1) {
                held_of[tid] = q.held;
                len_of[tid] = q.len;
            }
            A.first_pop[b] = (int)min(x.want, room);
            x = plus(x, asked(q), most);
            A.granted[b] = change;
            A.starts[b + 1] = (int)(ok ? x.grow : got_rows);
            if (change != 0)
                A.lens[b] = q.len + change;
        });
    }
    if (tid == 0) {
        A.starts[0] = 0;
        A.first_pop[A.B] = (int)room;
        A.n_free[0] = (int)(room - got_pages);
    }
    if constexpr (EACH == 1) {
        if (!with_rows)
            return;
        __syncthreads();
        for (int r = tid; r < A.rows; r += NT) {
            if (r >= (int)got_rows) {
                no_row(A, r);
                continue;
            }
            const int b = above([&](int i) { return sums[i + 1].grow; }, A.B, r);
            row(A, r, b, len_of[b] + r - (int)sums[b].grow, held_of[b], (int)sums[b].want, (int)room);
        }
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
            const int b = first + above([&](int i) { return ends[first + i]; }, last - first + 1, r);    // no load for one
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
    A.each = (int)nma::ceil_div(p.B, nms::kPlanThreads);
    hipStream_t s = static_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    // Few sequences need no block of 16 waves that wait for each other (32 sequences and rows, us with
    // 64 / 1024 threads: 2.7 / 9.8).
    const int threads = p.B <= 64 && rows <= 256 ? 64 : p.B <= 256 ? 256 : 1024;
    const bool with_rows = A.each == 1 && rows <= nms::kPlanRows * threads / nms::kPlanThreads;
    const auto plan = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(1), dim3(threads), 0, s, A, with_rows ? 1 : 0);
    };
    if (threads == 64)
        plan(plan_kernel<64, 1>);
    else if (threads == 256)
        plan(plan_kernel<256, 1>);
    else if (A.each == 1)
        plan(plan_kernel<nms::kPlanThreads, 1>);
    else if (A.each <= 4)
        plan(plan_kernel<nms::kPlanThreads, 4>);
    else
        plan(plan_kernel<nms::kPlanThreads, 0>);
    if (!with_rows && rows > 0)
        hipLaunchKernelGGL(rows_kernel, flat_grid(nma::ceil_div(rows, kRowsBlock)), dim3(kRowsBlock), 0, s, A);
    return hipGetLastError() == hipSuccess ? NM_OK : NM_ERR_HIP;
}
