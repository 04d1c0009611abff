// Pages and slots for sequences that grow or shrink.
//
// Bound by latency: a step touches a few numbers a sequence.  One workgroup does the stack and the table: of 1024
// sequences at a time, a lane each, the sums over the sequences before, then the pages, several a lane -- each
// finds its sequence by bisection of those sums, between the sequences of every 64th page.  Returned pages are all
// on the stack before the first is taken, and how many there are decides where each goes, so they are gone through
// twice.  Each wave has one stretch of them, so that it counts and places without a word to the others but its
// count, and kAtOnce pages a lane, whose bisections and loads are under way together (with one a lane and a sum
// over all lanes for each 1024 pages, a step that returns 16 thousand pages and takes 12 thousand needed 61 us, now
// 26). The new tokens' slots follow in the same workgroup while they are few, else in a kernel of their own, whose
// workgroups do not wait for each other.
#include "step_internal.h"

namespace tcm {

namespace {

constexpr int kLanes = 1024, kWaves = kLanes / 64;
// Up to this many tokens the planning workgroup writes the slots itself
constexpr int kFewTokens = 8192;
constexpr int kAtOnce = 8;  // pages of a lane

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
    int o = 0;
    for (int step = n > 1 ? 1 << (31 - __builtin_clz(n - 1)) : 0; step > 0; step /= 2)
        if (o + step < n && before[o + step] <= i) o += step;
    return o;
}
// The same for the numbers 64 u + lane from i0 on (past the end: the last one): lanes find those of every 64th
// number, and the others look between them, where there is mostly one sequence or two.
__device__ __forceinline__ void owners(const int64_t* before, int n, int64_t i0, int64_t end, int64_t* i, int* o) {
    const int lane = threadIdx.x & 63;
    const int edge = owner(before, n, min(i0 + 64 * min(lane, kAtOnce), end - 1));
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
        i[u] = min(i0 + 64 * u + lane, end - 1);
        const int lo = __builtin_amdgcn_readlane(edge, u), hi = __builtin_amdgcn_readlane(edge, u + 1);
        o[u] = lo + owner(before + lo, hi - lo + 1, i[u]);
    }
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
    const int lane = tid & 63, wave = tid >> 6;
    // the sums of the sequences from b0 on; all of their pages
    auto drops = [&](int b0) {
        const Span s = span_of(a, b0 + tid);
        const int old = pages_for(a, s.from), now = pages_for(a, s.to);
        int64_t all;
        const int64_t mine = scan(max(old - now, 0), red, all);
        before[tid] = mine;
        first[tid] = now;
        __syncthreads();
        return all;
    };
    // Goes through this wave's pages of them, in order: put(page or -1, entry or NULL, valid ones of the wave
    // before it); returns its valid ones.
    auto sweep = [&](int b0, int64_t all, auto put) {
        const int n = min(a.B - b0, kLanes);
        const int64_t per = (all + kLanes - 1) / kLanes * 64, end = min(all, (wave + 1) * per);
        int64_t seen = 0;
        for (int64_t i0 = wave * per; i0 < end; i0 += 64 * kAtOnce) {
            int64_t i[kAtOnce];
            int o[kAtOnce], page[kAtOnce];
            int32_t* entry[kAtOnce];
            owners(before, n, i0, end, i, o);
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                entry[u] = a.table + (b0 + o[u]) * a.table_stride + first[o[u]] + (int)(i[u] - before[o[u]]);
                page[u] = *entry[u];
            }
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const bool in = i0 + 64 * u + lane < end, is = in && (uint32_t)page[u] < (uint32_t)a.pages;
                const uint64_t valid = __ballot(is);
                put(is ? page[u] : -1, in ? entry[u] : nullptr, seen + __popcll(valid & ((1ull << lane) - 1)));
                seen += __popcll(valid);
            }
        }
        return seen;
    };
    // the waves' counts: those before this one's, and all
    auto meet = [&](int64_t mine, int64_t& total) {
        if (lane == 0) red[wave] = mine;
        __syncthreads();
        int64_t at = 0;
        total = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            at += w < wave ? red[w] : 0;
            total += red[w];
        }
        return at;
    };
    const auto nothing = [](int, int32_t*, int64_t) {};
    // (scan()'s barriers keep a sum from being overwritten before it is read)
    int64_t returned = 0, dropped = 0, all = 0, valid = 0, at = 0;
    for (int b0 = 0; b0 < a.B; b0 += kLanes) {
        all = drops(b0);
        at = meet(sweep(b0, all, nothing), valid);
        dropped += all;
        returned += valid;
    }
    int64_t seen = 0;
    for (int b0 = 0; b0 < a.B && dropped > 0; b0 += kLanes) {
        if (a.B > kLanes) {  // (else the sums and counts are there)
            all = drops(b0);
            at = meet(sweep(b0, all, nothing), valid);
        }
        const int64_t top = count + returned - 1 - seen - at;
        sweep(b0, all, [&](int page, int32_t* entry, int64_t r) {
            if (page >= 0 && top - r < a.capacity) a.stack[top - r] = page;
            if (entry) *entry = -1;
        });
        seen += valid;
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
        const int64_t per = (need + kLanes - 1) / kLanes * 64, end = min(need, (wave + 1) * per);
        for (int64_t i0 = wave * per; i0 < end; i0 += 64 * kAtOnce) {
            int64_t i[kAtOnce];
            int o[kAtOnce], page[kAtOnce];
            owners(before, n, i0, end, i, o);
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const int64_t from_top = top - 1 - taken - i[u];
                page[u] = from_top >= 0 ? a.stack[from_top] : -1;
            }
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u)  // (past the end: the last one's again)
                a.table[(b0 + o[u]) * a.table_stride + first[o[u]] + (int)(i[u] - before[o[u]])] = page[u];
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
