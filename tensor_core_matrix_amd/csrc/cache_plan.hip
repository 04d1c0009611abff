// Pages and slots for sequences that grow or shrink.
//
// Bound by latency: a step touches a few numbers a sequence.  One workgroup does the stack and
// the table: of 1024 sequences at a time, a lane each, the sums over the sequences before, then
// the pages, one a lane -- each finds its sequence by bisection of those sums.  Returned
// pages are all on the stack before the first is taken, so sequences are gone through twice.
// The new tokens' slots follow in the same workgroup while they are few, else in a kernel of
// their own, whose workgroups do not wait for each other.
#include "step_internal.h"

namespace tcm {

namespace {

constexpr int kLanes = 1024, kWaves = kLanes / 64;
// Up to this many tokens the planning workgroup writes the slots itself
constexpr int kFewTokens = 8192;

__device__ __forceinline__ int page_of(const PlanArgs& a, int key) {
    return a.page_shift >= 0 ? key >> a.page_shift : key / a.page_size;
}
__device__ __forceinline__ int pages_for(const PlanArgs& a, int keys) { return keys > 0 ? page_of(a, keys - 1) + 1 : 0; }

// Sum of x over the lanes before this one; `total` over all.  Two barriers.
__device__ __forceinline__ int64_t scan(int64_t x, int64_t* red, int64_t& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t s = x;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int64_t y = __shfl_up(s, d);
        if (lane >= d) s += y;
    }
    __syncthreads();  // (red is free)
    if (lane == 63) red[wave] = s;
    __syncthreads();
    int64_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        before += w < wave ? red[w] : 0;
        total += red[w];
    }
    return before + s - x;
}

// The last of the n sequences whose sum of those before it is at most i (sums do not fall)
__device__ __forceinline__ int owner(const int64_t* before, int n, int64_t i) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (before[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

struct Span {
    int from, to;  // keys before and after
};
__device__ __forceinline__ Span span_of(const PlanArgs& a, int b) {
    Span s = {0, 0};
    if (b < a.B) {
        const int room = a.width * a.page_size;
        s.from = min(max(a.lengths[b], 0), room);
        s.to = (int)min(max((int64_t)s.from + a.change[b], (int64_t)0), (int64_t)room);
    }
    return s;
}

// Slot and position of token t of sequence b, the i-th new one from key `from` on
__device__ __forceinline__ void write_token(const PlanArgs& a, int t, int b, int key) {
    const int e = page_of(a, key);
    const int page = a.table[b * a.table_stride + e];
    if (a.slots) a.slots[t] = (uint32_t)page < (uint32_t)a.pages ? page * a.page_size + (key - e * a.page_size) : -1;
    if (a.positions) a.positions[t] = key;
}
__device__ __forceinline__ void write_none(const PlanArgs& a, int t) {
    if (a.slots) a.slots[t] = -1;
    if (a.positions) a.positions[t] = 0;
}

__global__ __launch_bounds__(kLanes) void plan_kernel(PlanArgs a) {
    __shared__ int64_t red[kWaves];
    __shared__ int64_t before[kLanes];
    __shared__ int64_t tokens[kLanes];
    __shared__ int first[kLanes], from[kLanes];
    const int tid = threadIdx.x;
    const int count = min(max(*a.count, 0), a.capacity);

    // Pages that go back.  How many there are decides where each goes, so they are counted first.
    int64_t returned = 0;
    for (int pass = 0; pass < 2; ++pass) {
        int64_t seen = 0, dropped = 0;
        for (int b0 = 0; b0 < a.B; b0 += kLanes) {
            const Span s = span_of(a, b0 + tid);
            const int old = pages_for(a, s.from), now = pages_for(a, s.to);
            int64_t all;
            const int64_t mine = scan(max(old - now, 0), red, all);
            before[tid] = mine;
            first[tid] = now;
            __syncthreads();
            const int n = min(a.B - b0, kLanes);
            for (int64_t i0 = 0; i0 < all; i0 += kLanes) {
                int page = -1;
                int32_t* entry = nullptr;
                if (i0 + tid < all) {
                    const int o = owner(before, n, i0 + tid);
                    entry = a.table + (b0 + o) * a.table_stride + first[o] + (int)(i0 + tid - before[o]);
                    page = *entry;
                }
                const bool is = (uint32_t)page < (uint32_t)a.pages;
                int64_t valid;
                const int64_t r = seen + scan(is, red, valid);
                if (pass == 1) {
                    const int64_t at = count + returned - 1 - r;
                    if (is && at < a.capacity) a.stack[at] = page;
                    if (entry) *entry = -1;
                }
                seen += valid;
            }
            dropped += all;
            __syncthreads();  // (`before` and `first` are free)
        }
        returned = seen;
        if (dropped == 0) break;
    }
    __syncthreads();  // (the stack is whole)
    const int64_t top = min((int64_t)count + returned, (int64_t)a.capacity);

    // Pages that are taken, and tokens
    int64_t taken = 0, written = 0;
    for (int b0 = 0; b0 < a.B; b0 += kLanes) {
        const int b = b0 + tid;
        const Span s = span_of(a, b);
        const int old = pages_for(a, s.from), now = pages_for(a, s.to);
        int64_t need, fresh;
        const int64_t mine = scan(max(now - old, 0), red, need);
        const int64_t token = written + scan(max(s.to - s.from, 0), red, fresh);
        before[tid] = mine;
        tokens[tid] = token;
        first[tid] = old;
        from[tid] = s.from;
        if (b < a.B) {
            a.starts[b] = (int)min(token, (int64_t)INT32_MAX);
            a.lengths[b] = s.to;
        }
        __syncthreads();
        const int n = min(a.B - b0, kLanes);
        for (int64_t i = tid; i < need; i += kLanes) {
            const int o = owner(before, n, i);
            const int64_t at = top - 1 - taken - i;
            a.table[(b0 + o) * a.table_stride + first[o] + (int)(i - before[o])] = at >= 0 ? a.stack[at] : -1;
        }
        __syncthreads();
        if (a.T <= kFewTokens)
            for (int64_t t = written + tid; t < min(written + fresh, (int64_t)a.T); t += kLanes) {
                const int o = owner(tokens, n, t);
                write_token(a, (int)t, b0 + o, from[o] + (int)(t - tokens[o]));
            }
        taken += need;
        written += fresh;
        __syncthreads();  // (the arrays are free)
    }
    if (a.T <= kFewTokens)
        for (int64_t t = written + tid; t < a.T; t += kLanes) write_none(a, (int)t);
    if (tid == 0) {
        a.starts[a.B] = (int)min(written, (int64_t)INT32_MAX);
        *a.count = (int)max(top - taken, (int64_t)0);
        if (a.missing) *a.missing = (int)max(taken - top, (int64_t)0);
    }
}

// Slots and positions of many tokens, after plan_kernel; starts are all there, as int32.
__global__ __launch_bounds__(256) void slots_kernel(PlanArgs a) {
    const int t = blockIdx.x * 256 + threadIdx.x;
    if (t >= a.T) return;
    if (t >= a.starts[a.B]) return write_none(a, t);
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.starts[mid] <= t) lo = mid;
        else hi = mid;
    }
    // its new tokens are the last of its keys
    const int n = a.starts[lo + 1] - a.starts[lo];
    write_token(a, t, lo, a.lengths[lo] - n + (t - a.starts[lo]));
}

}  // namespace

hipError_t launch_cache_plan(const PlanArgs& a, hipStream_t st) {
    hipLaunchKernelGGL(plan_kernel, dim3(1), dim3(kLanes), 0, st, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.T <= kFewTokens || !(a.slots || a.positions)) return e;
    hipLaunchKernelGGL(slots_kernel, dim3((a.T + 255) / 256), dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace tcm
