// paged_cache.cu -- bookkeeping and writes of a paged key/value cache.
//
// page_slots: from the tokens a request holds (ctx_lens) and the new ones it brings
// (cu_q), the pages it needs, taken from a free list in request order, and for every new token
// its position and its slot (page * page_size + row).  One launch, no atomics: every block sums
// the pages taken by the requests before its own, so the outcome depends on the lengths alone.
//   need_n = ceil((ctx_n + new_n) / page_size),  have_n = ceil(ctx_n / page_size),
//            both max_pages at most: a page without a column stays in the free list
//   first_n = free_start + sum_{m < n} (need_m - have_m)
//   table[n][have_n + i] = free_pages[first_n + i]       for i < need_n - have_n
// The blocks of the first part write table columns >= have_n, those of the second read columns
// < have_n and the free list, so the parts need no order.  Every block looks at the lengths of all
// requests first: if any does not fit, no block hands anything out.  Bound by latency: a block reads the
// lengths of all requests (coalesced) and makes one or two dependent look-ups: 2.8 us for 8
// requests of a token each, 10.1 us for 1024 of up to 128 (9.9 without a look at those behind it).
//
// paged_write: rows of K and V to their slots, 16 bytes per access; bound by DRAM bandwidth:
// 16384 tokens of H_kv = 8, d = 128, bf16 (134 MB moved) take 20 us (6.7 TB/s).  Two and four
// pieces in flight per thread took 20.2 and 24.2 us.
#include "packed.cuh"
#include "paged_cache.cuh"

namespace fa {
namespace {

constexpr int kT = 256;

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

struct Req {
    int ctx, fresh, have, taken;
};

// One request's numbers, for lengths that fit.
__device__ __forceinline__ Req request(const PageSlots& a, int ctx, int fresh) {
    const int have = min(ceil_div(ctx, a.page_size), a.max_pages);
    return {ctx, fresh, have, min(ceil_div(ctx + fresh, a.page_size), a.max_pages) - have};
}
__device__ __forceinline__ Req request(const PageSlots& a, int n) {
    return request(a, a.ctx_lens[n], a.cu_q[n + 1] - a.cu_q[n]);
}

// What a block needs to know of all requests, in one pass over their lengths.
struct Before {
    int count, taken;  // requests before the block's own, and the pages they take
    int bad;           // whether the lengths of some request, before or behind, do not fit
};

// is_before(n, end of n's rows): whether request n comes before the block's own.
template <typename F>
__device__ __forceinline__ Before look_over(const PageSlots& a, Before* sums, F is_before) {
    Before b = {0, 0, 0};
#pragma unroll 4
    for (int n = threadIdx.x; n < a.N; n += kT) {
        const int c0 = a.cu_q[n], c1 = a.cu_q[n + 1], ctx = a.ctx_lens[n];
        if (!(c0 >= 0 && c1 >= c0 && c1 <= a.T && ctx >= 0 && ctx <= (1 << 30))) {
            b.bad = 1;
        } else if (is_before(n, c1)) {
            ++b.count;
            b.taken += request(a, ctx, c1 - c0).taken;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        b.count += __shfl_xor_sync(0xffffffffu, b.count, o);
        b.taken += __shfl_xor_sync(0xffffffffu, b.taken, o);
        b.bad |= __shfl_xor_sync(0xffffffffu, b.bad, o);
    }
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = b;
    __syncthreads();
    b = {0, 0, 0};
#pragma unroll
    for (int w = 0; w < kT / 32; ++w) {
        b.count += sums[w].count;
        b.taken += sums[w].taken;
        b.bad |= sums[w].bad;
    }
    return b;
}

__device__ __forceinline__ int block_sum(int v, int* sums) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = v;
    __syncthreads();
    int s = 0;
#pragma unroll
    for (int w = 0; w < kT / 32; ++w) s += sums[w];
    return s;
}

// Exclusive scan over the block.
__device__ __forceinline__ int block_scan(int v, int* sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = s;
    __syncthreads();
    int before = 0;
#pragma unroll
    for (int w = 0; w < kT / 32; ++w) before += w < warp ? sums[w] : 0;
    return before + s - v;
}

// Page of the free list, or -1 when it has run out.
__device__ __forceinline__ int take(const PageSlots& a, long long i) {
    if (i >= 0 && i < a.n_free) return a.free_pages[i];
    return -1;
}

__global__ void __launch_bounds__(kT) page_slots_kernel(const PageSlots a, int req_blocks) {
    __shared__ int s_sum[kT / 32];
    __shared__ int s_cu[kT + 1], s_ctx[kT], s_first[kT];
    __shared__ Before s_before[kT / 32];
    const int tid = threadIdx.x;
    const long long start = *a.free_start;
    if ((int)blockIdx.x < req_blocks) {
        // ---- requests: table entries, lengths, where the free list goes on
        const int r0 = blockIdx.x * kT, n = r0 + tid;
        const Before b = look_over(a, s_before, [&](int m, int) { return m < r0; });
        if (b.bad) {  // nothing is handed out: the requests hold what they held
            if (n < a.N) a.seq_lens[n] = a.ctx_lens[n];
            if (n == 0) {
                *a.free_next = (int)start;
                atomicOr(a.err, kErrLengths);
            }
            return;
        }
        Req r = {0, 0, 0, 0};
        if (n < a.N) r = request(a, n);
        const int at = b.taken + block_scan(r.taken, s_sum);
        unsigned e = 0u;
        const bool last = n == a.N - 1;
        if (n < a.N) a.seq_lens[n] = r.ctx + r.fresh;
        if (last) *a.free_next = (int)(start + at + r.taken);
        if (__syncthreads_or(last && start + at + r.taken > a.n_free)) {
            // the list ran out: how far it falls short of all that the tokens ask for
            int asked = 0;
            for (int m = tid; m < a.N; m += kT) {
                const Req q = request(a, m);
                asked += ceil_div(q.ctx + q.fresh, a.page_size) - ceil_div(q.ctx, a.page_size);
            }
            asked = block_sum(asked, s_sum);
            if (last) *a.free_next = (int)(start + asked);
        }
        // one warp writes one request's entries at a time
        s_first[tid] = at;
        s_cu[tid] = r.have;
        s_ctx[tid] = r.taken;
        __syncthreads();
        const int lane = tid & 31;
        for (int q = tid >> 5; q < kT; q += kT / 32) {
            if (r0 + q >= a.N) break;
            int* row = a.table + (size_t)(r0 + q) * a.max_pages;
            for (int i = lane; i < s_ctx[q]; i += 32) {
                const int col = s_cu[q] + i;
                const int id = take(a, start + s_first[q] + i);
                if (id < 0) e |= kErrPool;
                row[col] = id;
            }
        }
        if (e) atomicOr(a.err, e);
        return;
    }
    // ---- tokens: position and slot of rows [t0, t0 + kT)
    const int t0 = (blockIdx.x - req_blocks) * kT, t = t0 + tid;
    // the first request that ends behind t0, and the pages taken before it
    const Before b = look_over(a, s_before, [&](int, int end) { return end <= t0; });
    int n0 = b.count, before = b.taken;
    const int t_end = min(t0 + kT, a.T);
    bool done = t >= a.T;
    if (t < a.T) {
        a.slots[t] = -1;  // rows behind the last request
        a.positions[t] = -1;
    }
    if (b.bad) return;  // no row has a slot
    // windows of kT requests until one ends behind the block's last token
    while (n0 < a.N) {
        const int n = n0 + tid;
        Req r = {0, 0, 0, 0};
        if (n < a.N) r = request(a, n);
        const int at = before + block_scan(r.taken, s_sum);
        const int live = min(kT, a.N - n0);
        s_first[tid] = at;
        s_ctx[tid] = r.ctx;
        if (n < a.N) s_cu[tid] = a.cu_q[n];
        if (tid == 0) s_cu[live] = a.cu_q[n0 + live];
        __syncthreads();
        if (!done && t >= s_cu[0] && t < s_cu[live]) {
            done = true;
            int lo = 0, hi = live;  // largest lo with s_cu[lo] <= t
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_cu[mid] <= t)
                    lo = mid;
                else
                    hi = mid;
            }
            const int pos = s_ctx[lo] + (t - s_cu[lo]);
            if (pos >= 0) {
                const int col = pos / a.page_size, have = ceil_div(s_ctx[lo], a.page_size);
                int id = -1;
                if (col < a.max_pages)
                    id = col < have ? a.table[(size_t)(n0 + lo) * a.max_pages + col]
                                    : take(a, start + s_first[lo] + (col - have));
                a.positions[t] = pos;
                if (id >= 0) a.slots[t] = (long long)id * a.page_size + pos % a.page_size;
                else atomicOr(a.err, kErrPool);
            }
        }
        const bool more = s_cu[live] < t_end;
        before += block_sum(r.taken, s_sum);
        n0 += kT;
        if (!more) break;
    }
}

__global__ void __launch_bounds__(kT) paged_write_kernel(const PagedWrite a) {
    // e counts the 16-byte pieces of the T rows; both tensors' piece e belong to one thread
    const int per = a.H_kv * a.cpr;
    const long long total = (long long)a.T * per;
    const long long stride = (long long)gridDim.x * kT;
    for (long long e = (long long)blockIdx.x * kT + threadIdx.x; e < total; e += stride) {
        const int t = (int)(e / per), c = (int)(e - (long long)t * per);
        const int h = c / a.cpr, x = c - h * a.cpr;
        const long long slot = a.slots[t];
        if (slot < 0) continue;  // a padding row
        const long long pg = slot / a.page_size, row = slot - pg * a.page_size;
        if (pg >= a.pages) {
            if (c == 0) atomicOr(a.err, kErrPage);
            continue;
        }
        const uint4* ks = reinterpret_cast<const uint4*>(static_cast<const char*>(a.K) + t * a.k.tok + h * a.k.head);
        const uint4* vs = reinterpret_cast<const uint4*>(static_cast<const char*>(a.V) + t * a.v.tok + h * a.v.head);
        const uint4 kv = __ldcs(ks + x), vv = __ldcs(vs + x);
        reinterpret_cast<uint4*>(static_cast<char*>(a.K_cache) + pg * a.kc_page + row * a.kc.tok + h * a.kc.head)[x] = kv;
        reinterpret_cast<uint4*>(static_cast<char*>(a.V_cache) + pg * a.vc_page + row * a.vc.tok + h * a.vc.head)[x] = vv;
    }
}

}  // namespace

cudaError_t launch_page_slots(const PageSlots& a, cudaStream_t st) {
    const int rb = (a.N + kT - 1) / kT, tb = (a.T + kT - 1) / kT;
    page_slots_kernel<<<rb + tb, kT, 0, st>>>(a, rb);
    return cudaGetLastError();
}

cudaError_t launch_paged_write(const PagedWrite& a, cudaStream_t st) {
    const long long total = (long long)a.T * a.H_kv * a.cpr;
    long long grid = (total + kT - 1) / kT;
    if (grid > 152 * 32) grid = 152 * 32;
    paged_write_kernel<<<(unsigned)grid, kT, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace fa
