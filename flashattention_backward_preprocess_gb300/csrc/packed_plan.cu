// packed_plan.cu -- work plans of the packed and paged operators, built on the device from the
// sequence lengths so that no call has to read them back.  One block plans (prefix sums over
// sequences and units, a few microseconds); the other blocks fill the output rows that belong
// to no sequence when the caller asked for that.
#include "packed.cuh"

namespace fa {
namespace {

constexpr int kPlanThreads = 1024;

template <typename V>
__device__ __forceinline__ V warp_incl_scan(V v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const V u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}

// Exclusive scan over the block; *total gets the block's sum.  Ends with a barrier.
template <typename V>
__device__ __forceinline__ V block_excl_scan(V v, V* sums, V* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (int)blockDim.x >> 5;
    const V incl = warp_incl_scan(v);
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const V s = lane < warps ? sums[lane] : V(0);
        const V si = warp_incl_scan(s);
        sums[lane] = si - s;
        if (lane == 31) sums[32] = si;
    }
    __syncthreads();
    const V r = sums[warp] + incl - v;
    *total = sums[32];
    __syncthreads();
    return r;
}

struct Seq {
    int q0, nq, k0, nk;
};

// Lengths of sequence n; false if they do not fit the tensors.
__device__ __forceinline__ bool seq_at(const PackedFwd& a, int n, Seq& s) {
    const int q0 = a.cu_q[n], q1 = a.cu_q[n + 1];
    bool ok = q0 >= 0 && q1 >= q0 && q1 <= a.T_q;
    s.q0 = q0;
    s.nq = ok ? q1 - q0 : 0;
    if (a.cu_k != nullptr) {
        const int k0 = a.cu_k[n], k1 = a.cu_k[n + 1];
        const bool okk = k0 >= 0 && k1 >= k0 && k1 <= a.T_k;
        s.k0 = k0;
        s.nk = okk ? k1 - k0 : 0;
        ok = ok && okk;
    } else {
        const int nk = a.seq_lens[n];
        // longer than its table, or than positions are kept for, is refused
        const bool okk = nk >= 0 && nk <= (1 << 28) && nk <= (long long)a.max_pages * a.page_size;
        s.k0 = 0;
        s.nk = okk ? nk : 0;
        ok = ok && okk;
    }
    return ok;
}

// Largest n with first[n] <= u (first is non-decreasing, first[N] > u).
__device__ __forceinline__ int find_seq(const int* first, int N, int u) {
    int lo = 0, hi = N;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (first[mid] <= u)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

constexpr int kSmemSeqs = 4096;  // sequences whose unit offsets are also kept in shared memory

template <typename T>
__device__ void fill_rows(const PackedFwd& a) {
    // rows before the first and behind the last sequence: O = 0, LSE = -inf
    const int lo = a.cu_q[0], hi = a.cu_q[a.N];
    if (lo < 0 || hi < lo || hi > a.T_q) return;  // reported by the planning block
    const long long rows = (long long)(lo + a.T_q - hi) * a.H;
    const int per = a.d * (int)sizeof(T) / 16;
    const long long step = (long long)(gridDim.x - 1) * blockDim.x;
    for (long long e = (long long)(blockIdx.x - 1) * blockDim.x + threadIdx.x; e < rows * per; e += step) {
        const long long r = e / per;
        const int t = (int)(r / a.H), h = (int)(r % a.H), c = (int)(e % per);
        const int tok = t < lo ? t : t - lo + hi;
        T* dst = static_cast<T*>(a.O) + tok * a.o.tok + h * a.o.head + c * (16 / (int)sizeof(T));
        *reinterpret_cast<uint4*>(dst) = make_uint4(0u, 0u, 0u, 0u);
        if (c == 0) a.LSE[(size_t)h * a.T_q + tok] = -INFINITY;
    }
}

__global__ void __launch_bounds__(kPlanThreads) fwd_plan_kernel(const PackedFwd a, const FwdGeom g, const FwdPlan p) {
    ptx::griddep_launch_dependents();
    if (blockIdx.x > 0) {
        if (a.dtype == FA_F32)
            fill_rows<float>(a);
        else
            fill_rows<__half>(a);
        return;
    }
    __shared__ int s_first[kSmemSeqs + 1];
    __shared__ int s_isum[33];
    __shared__ long long s_lsum[33];
    const int tid = threadIdx.x;
    int* first = a.N <= kSmemSeqs ? s_first : p.seq_units;

    // units of each sequence
    int U = 0;
    bool bad = false;
    for (int n0 = 0; n0 < a.N; n0 += kPlanThreads) {
        const int n = n0 + tid;
        int units = 0;
        if (n < a.N) {
            Seq s;
            if (!seq_at(a, n, s)) bad = true;
            units = (s.nq + g.tpt - 1) / g.tpt;
        }
        int total;
        const int at = block_excl_scan(units, s_isum, &total);
        if (n < a.N) first[n] = U + at;
        U += total;
    }
    if (tid == 0) first[a.N] = U;
    if (__syncthreads_or(bad)) {  // lengths that do not fit the tensors: nothing is computed
        if (tid == 0) atomicOr(a.err, kErrLengths);
        U = 0;
    }

    // tiles of each unit and their places on the axis of positions
    long long W = 0;
    for (int u0 = 0; u0 < U; u0 += kPlanThreads) {
        const int u = u0 + tid;
        long long cost = 0;
        if (u < U) {
            const int n = find_seq(first, a.N, u);
            Seq s;
            seq_at(a, n, s);
            const int i0 = (u - first[n]) * g.tpt;
            FwdTile t;
            t.n = n;
            t.q_tok = s.q0 + i0;
            t.n_tok = min(g.tpt, s.nq - i0);
            t.pos0 = i0 + s.nk - s.nq;
            t.k_base = s.k0;
            t.S_k = s.nk;
            Shape sh;
            sh.S_q = s.nq;
            sh.S_k = s.nk;
            sh.causal = a.causal;
            sh.window = a.window;
            int lo, hi;
            key_range(sh, i0, i0 + t.n_tok, lo, hi);
            t.n_first = hi > lo ? lo / g.bn : 0;
            t.n_cnt = hi > lo ? (hi + g.bn - 1) / g.bn - t.n_first : 0;
            p.tile[u] = t;
            cost = (long long)max(t.n_cnt, 1) * g.heads;
        }
        long long total;
        const long long at = block_excl_scan(cost, s_lsum, &total);
        if (u < U) p.base[u] = W + at;
        W += total;
    }

    // equal shares, and the unit each CTA starts in
    long long chunk = (W + g.ctas - 1) / g.ctas;
    if (chunk < g.min_chunk) chunk = g.min_chunk;
    if (tid == 0) {
        p.head[0] = W;
        p.head[1] = chunk;
    }
    for (int c = tid; c < g.ctas; c += kPlanThreads) p.done[c] = 0u;
    for (int u = tid; u < U; u += kPlanThreads) {
        const long long b = p.base[u];
        const long long e = b + (long long)max(p.tile[u].n_cnt, 1) * g.heads;
        for (long long c = (b + chunk - 1) / chunk; c * chunk < e; ++c) p.start[c] = u;
    }
}

}  // namespace

cudaError_t launch_fwd_plan(const PackedFwd& a, const FwdGeom& g, const FwdPlan& p, cudaStream_t st) {
    fwd_plan_kernel<<<a.fill ? 33 : 1, kPlanThreads, 0, st>>>(a, g, p);
    return cudaGetLastError();
}

}  // namespace fa
