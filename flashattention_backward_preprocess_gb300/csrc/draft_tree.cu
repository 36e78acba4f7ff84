// draft_tree.cu -- trees of drafted tokens over a paged cache: who sees whom, and what is left of
// the step once the accepted tokens are known.
//
// tree_mask: node i of a request names its parent, an earlier node or -1 (it follows the cached
// tokens).  Bit k of node i's mask: k is i or an ancestor of i.  Position: tokens cached before the
// step + number of ancestors.  A thread walks up from its node; the parents' numbers fall, so the
// walk ends and the mask's words are finished from the last to the first.
//
// paged_keep: rows ctx + path[i] of the cache to ctx + i, for the accepted nodes path[0] < path[1]
// < ... of each request, in every layer.  A thread takes the same 16 bytes of all rows in order:
// path[i] >= i, so a row is never written before it has been read, and no two threads share bytes.
//
// page_trim: lengths ctx + count, and the pages that only dropped tokens used back to the free
// list, in front of its first unused entry, request after request.  The entries written are ones
// that were used up, the table keeps its stale columns (nothing reads behind a request's last page),
// so the call only writes what it does not read and may be run again.  By path it leaves the requests alone
// that paged_keep leaves alone (step_fits, path_fits): their tokens all stay, the other requests are trimmed.
//
// All three are bound by latency, a few dependent look-ups beside the launch: masks of 32 trees of 8 to
// 64 tokens 4 us, rows of 64 requests in 16 layers 10 us, pages of 64 requests 5 us.
#include "packed.cuh"
#include "paged_cache.cuh"

namespace fa {
namespace {

constexpr int kT = 128;

__device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

__global__ void __launch_bounds__(kT) tree_mask_kernel(const TreeMask a) {
    bool bad = false;
    for (int n = threadIdx.x; n < a.N; n += kT) {
        const int c0 = a.cu_q[n], c1 = a.cu_q[n + 1], ctx = a.ctx_lens[n];
        bad |= !(c0 >= 0 && c1 >= c0 && c1 <= a.T && ctx >= 0 && ctx <= (1 << 28) - (c1 - c0));
    }
    bad = __syncthreads_or(bad);
    const int t = blockIdx.x * kT + threadIdx.x;
    if (bad && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.err, kErrLengths);
    if (t >= a.T) return;
    unsigned long long* out = a.tree + (size_t)t * a.words;
    if (bad || t < a.cu_q[0] || t >= a.cu_q[a.N]) {  // a row of no request
        for (int w = 0; w < a.words; ++w) out[w] = 0ull;
        a.positions[t] = -1;
        return;
    }
    const int n = find_seq(a.cu_q, a.N, t);
    const int c0 = a.cu_q[n], i = t - c0;
    bool wrong = i >= 64 * a.words;  // no bit of its own
    int w = a.words - 1, depth = 0;
    unsigned long long bits = 0ull;
    for (int node = i;;) {
        for (; w > node >> 6; --w) {
            out[w] = bits;
            bits = 0ull;
        }
        if (w == node >> 6) bits |= 1ull << (node & 63);
        const int up = a.parents[c0 + node];
        if (up < 0 || up >= node) {
            wrong |= up != -1;
            break;
        }
        node = up;
        ++depth;
    }
    for (; w >= 0; --w) {
        out[w] = bits;
        bits = 0ull;
    }
    a.positions[t] = a.ctx_lens[n] + depth;
    if (wrong) atomicOr(a.err, kErrTree);
}

// Whether a request's offsets, length and number of accepted tokens fit.
__device__ __forceinline__ bool step_fits(int c0, int c1, int T, int len, int count) {
    return c0 >= 0 && c1 >= c0 && c1 <= T && len >= c1 - c0 && len <= (1 << 28) && count >= 0 && count <= c1 - c0;
}
// Whether entry i of a request's path, of `fresh` new tokens, does.
__device__ __forceinline__ bool path_fits(const int* path, int i, int fresh) {
    const int p = path[i];
    return p >= 0 && p < fresh && (i == 0 || p > path[i - 1]);
}

// Block: columns [blockIdx.y * kT, + kT) of a tensor's row in layer blockIdx.z / 2, one request.
__global__ void __launch_bounds__(kT) paged_keep_kernel(const __grid_constant__ PagedKeep a) {
    constexpr int kBatch = 4;  // rows in flight
    const int n = blockIdx.x, layer = blockIdx.z >> 1;
    const bool is_v = blockIdx.z & 1;
    const int count = a.count[n], c0 = a.cu_q[n], c1 = a.cu_q[n + 1], len = a.seq_lens[n];
    if (count == 0) return;
    const bool first = blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0;
    if (!step_fits(c0, c1, a.T, len, count)) {
        if (first) atomicOr(a.err, kErrTree);
        return;
    }
    const int* path = a.path + c0;
    bool bad = false;
    for (int i = threadIdx.x; i < count; i += kT) bad |= !path_fits(path, i, c1 - c0);
    if (__syncthreads_or(bad)) {
        if (first) atomicOr(a.err, kErrTree);
        return;
    }
    const int c = blockIdx.y * kT + threadIdx.x;
    if (c >= a.H_kv * a.cpr) return;
    const int h = c / a.cpr, x = c - h * a.cpr, ctx = len - (c1 - c0);
    char* base = static_cast<char*>(is_v ? a.V[layer] : a.K[layer]) + (is_v ? a.vc.head : a.kc.head) * h + x * 16;
    const long long page_b = is_v ? a.vc_page : a.kc_page, row_b = is_v ? a.vc.tok : a.kc.tok;
    uint8_t* exps = is_v ? a.v_exp[layer] : a.k_exp[layer];
    const bool has_exp = exps != nullptr && x == 0;
    const int* row = a.table + (size_t)n * a.max_pages;
    bool lost = false;
    for (int i0 = 0; i0 < count; i0 += kBatch) {
        uint4 data[kBatch];
        uint8_t e[kBatch];
        int to[kBatch];  // page of the target, -1: stays where it is
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int i = i0 + b;
            to[b] = -1;
            if (i >= count) continue;
            const int p = path[i];
            if (p == i) continue;
            const int from = page_of(row, ctx + p, a.page_size, a.max_pages, a.pages, &lost);
            const int dst = page_of(row, ctx + i, a.page_size, a.max_pages, a.pages, &lost);
            if (from == a.pages || dst == a.pages) continue;
            to[b] = dst;
            const int in = (ctx + p) % a.page_size;
            data[b] = *reinterpret_cast<const uint4*>(base + from * page_b + in * row_b);
            if (has_exp) e[b] = exps[((long long)from * a.H_kv + h) * a.page_size + in];
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (to[b] < 0) continue;
            const int in = (ctx + i0 + b) % a.page_size;
            *reinterpret_cast<uint4*>(base + to[b] * page_b + in * row_b) = data[b];
            if (has_exp) exps[((long long)to[b] * a.H_kv + h) * a.page_size + in] = e[b];
        }
    }
    if (lost && first) atomicOr(a.err, kErrPage);
}

constexpr int kTrimT = 256;

__global__ void __launch_bounds__(kTrimT) page_trim_kernel(const PageTrim a) {
    __shared__ int s_sum[33];
    const int tid = threadIdx.x;
    const int start = *a.free_start;
    // with paths: what request n keeps, all it has where its numbers do not fit
    auto kept_alone = [&](int n) {
        const int c0 = a.cu_q[n], c1 = a.cu_q[n + 1], len = a.seq_lens[n], count = a.count[n];
        bool fits = step_fits(c0, c1, a.T, len, count);
        for (int i = 0; fits && i < count; ++i) fits = path_fits(a.path + c0, i, c1 - c0);
        if (!fits) atomicOr(a.err, kErrTree);
        return fits ? len - (c1 - c0) + count : len;
    };
    // columns [need, had) of request n's row are given back
    auto gone = [&](int n, int& need, int& had) {
        const int len = a.seq_lens[n];
        // (the first pass has written lens, by this thread, where there are paths)
        const int kept = a.by_path ? a.lens[n] : len - (a.cu_q[n + 1] - a.cu_q[n]) + a.count[n];
        if (a.by_path && kept == len) return 0;
        need = min(ceil_div(kept, a.page_size), a.max_pages);
        had = min(ceil_div(len, a.page_size), a.max_pages);
        int c = 0;
        for (int i = need; i < had; ++i) c += a.table[(size_t)n * a.max_pages + i] >= 0;
        return c;
    };
    bool bad = false;
    for (int n = tid; n < a.N; n += kTrimT) {
        if (a.by_path) {
            a.lens[n] = kept_alone(n);
            continue;
        }
        const int c0 = a.cu_q[n], c1 = a.cu_q[n + 1], len = a.seq_lens[n], count = a.count[n];
        bad |= !(c0 >= 0 && c1 >= c0 && len >= c1 - c0 && len <= (1 << 30) && count >= 0 && count <= c1 - c0);
    }
    bad = __syncthreads_or(bad);
    long long all = 0;
    if (!bad)
        for (int n0 = 0; n0 < a.N; n0 += kTrimT) {
            int need, had, total;
            block_excl_scan(n0 + tid < a.N ? gone(n0 + tid, need, had) : 0, s_sum, &total);
            all += total;
        }
    const long long next = (start < a.n_free ? start : a.n_free) - all;
    // more pages given back than were taken: none of them is entered
    const bool full = all > 0 && (next < 0 || start < 0);
    if (tid == 0) {
        *a.free_next = bad || full || all == 0 ? start : (int)next;
        if (bad) atomicOr(a.err, kErrLengths);
        if (full) atomicOr(a.err, kErrPool);
    }
    long long at0 = next;
    for (int n0 = 0; n0 < a.N; n0 += kTrimT) {
        const int n = n0 + tid;
        if (bad || full) {
            if (n < a.N && !a.by_path) a.lens[n] = bad ? a.seq_lens[n] : a.seq_lens[n] - (a.cu_q[n + 1] - a.cu_q[n]) + a.count[n];
            continue;
        }
        int need = 0, had = 0, total;
        const int mine = n < a.N ? gone(n, need, had) : 0;
        long long at = at0 + block_excl_scan(mine, s_sum, &total);
        at0 += total;
        if (n >= a.N) continue;
        if (!a.by_path) a.lens[n] = a.seq_lens[n] - (a.cu_q[n + 1] - a.cu_q[n]) + a.count[n];
        for (int i = need; i < had; ++i) {
            const int page = a.table[(size_t)n * a.max_pages + i];
            if (page >= 0) a.free_pages[at++] = page;
        }
    }
}

}  // namespace

cudaError_t launch_tree_mask(const TreeMask& a, cudaStream_t st) {
    tree_mask_kernel<<<(a.T + kT - 1) / kT, kT, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_paged_keep(const PagedKeep& a, cudaStream_t st) {
    const dim3 grid((unsigned)a.N, (unsigned)((a.H_kv * a.cpr + kT - 1) / kT), (unsigned)(2 * a.layers));
    paged_keep_kernel<<<grid, kT, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_page_trim(const PageTrim& a, cudaStream_t st) {
    page_trim_kernel<<<1, kTrimT, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace fa
