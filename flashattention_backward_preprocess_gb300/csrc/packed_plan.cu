// packed_plan.cu -- work plans of the packed and paged operators, built on the device from the
// sequence lengths so that no call has to read them back.  One block plans (prefix sums over
// sequences and units, a few microseconds); the other blocks fill the output rows that belong
// to no sequence when the caller asked for that.  Bound by latency: the forward plan of few
// sequences is made by every CTA of the forward itself instead (plan_self), which saves the
// launch; the backward's takes about 7 us of the 521 of ten sequences (11390 tokens).
#include "packed.cuh"
#include "tma_map.cuh"

namespace fa {
namespace {

constexpr int kPlanThreads = 1024;

constexpr int kSmemSeqs = 4096;  // sequences whose unit offsets are also kept in shared memory

// Lengths of sequence n of a backward; false (and empty) if they do not fit the tensors.
__device__ __forceinline__ bool seq_at(const PackedBwd& a, int n, Seq& s) {
    const int q0 = a.cu_q[n], q1 = a.cu_q[n + 1], k0 = a.cu_k[n], k1 = a.cu_k[n + 1];
    const bool ok = q0 >= 0 && q1 >= q0 && q1 <= a.T_q && k0 >= 0 && k1 >= k0 && k1 <= a.T_k;
    s.q0 = q0;
    s.nq = ok ? q1 - q0 : 0;
    s.k0 = k0;
    s.nk = ok ? k1 - k0 : 0;
    return ok;
}

// Whether the lengths of any sequence do not fit the tensors (asked by a whole block).
template <typename A>
__device__ __forceinline__ bool any_bad(const A& a) {
    bool bad = false;
    for (int n = threadIdx.x; n < a.N; n += blockDim.x) {
        Seq s;
        bad |= !seq_at(a, n, s);
    }
    return __syncthreads_or(bad);
}

__global__ void __launch_bounds__(kPlanThreads, 1) fwd_plan_kernel(const PackedFwd a, const FwdGeom g, const FwdPlan p) {
    ptx::griddep_launch_dependents();
    if (blockIdx.x > 0) {
        const long long first = (long long)(blockIdx.x - 1) * blockDim.x + threadIdx.x;
        const long long step = (long long)(gridDim.x - 1) * blockDim.x;
        const bool all = any_bad(a);  // nothing is computed then: no row is left unset
        if (a.dtype == FA_F32)
            fill_rows<float>(a, all, first, step);
        else
            fill_rows<__half>(a, all, first, step);
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
            if (past_table(a, s)) atomicOr(a.err, kErrLengths);
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
            FwdTile t;
            cost = (long long)make_tile(a, g, n, u - first[n], t) * g.heads;
            p.tile[u] = t;
        }
        long long total;
        const long long at = block_excl_scan(cost, s_lsum, &total);
        if (u < U) p.base[u] = W + at;
        W += total;
    }

    // equal shares, and the unit each CTA starts in
    const long long chunk = share_of(W, g);
    if (tid == 0) {
        p.head[0] = W;
        p.head[1] = chunk;
    }
    for (int u = tid; u < U; u += kPlanThreads) {
        const long long b = p.base[u];
        const long long e = b + (long long)(max(p.tile[u].n_cnt, 1) + g.overhead) * g.heads;
        for (long long c = (b + chunk - 1) / chunk; c * chunk < e; ++c) p.start[c] = u;
    }
}

// ---------------------------------------------------------------- backward
struct BwdMaps {
    CUtensorMap m[kSeqMaps];  // Q, dO, K, V, accumulator of the whole call
};

// The maps of sequence n: the call's, based at its first row and as long as the sequence.
__device__ __forceinline__ void write_map(CUtensorMap* dst, const CUtensorMap* src, uint32_t buf, uint32_t* buf_p,
                                          const void* base, int rows, int lane) {
    buf_p[lane] = reinterpret_cast<const uint32_t*>(src)[lane];
    __syncwarp();
    if (lane == 0) {
        asm volatile("tensormap.replace.tile.global_address.shared::cta.b1024.b64 [%0], %1;" ::"r"(buf),
                     "l"(reinterpret_cast<uint64_t>(base))
                     : "memory");
        asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 2, %1;" ::"r"(buf), "r"(rows)
                     : "memory");
    }
    __syncwarp();
    asm volatile(
        "tensormap.cp_fenceproxy.global.shared::cta.tensormap::generic.release.gpu.sync.aligned [%0], [%1], 128;" ::"l"(
            reinterpret_cast<uint64_t>(dst)),
        "r"(buf)
        : "memory");
    __syncwarp();
}

// rows [0, lo) and [hi, T) of a gradient
template <typename T>
__device__ void zero_rows(void* X, RowStride s, int heads, int d, int lo, int hi, int T_all, int part, int parts) {
    const int per = d * (int)sizeof(T) / 16;
    const long long n = (long long)(lo + T_all - hi) * heads * per;
    for (long long e = (long long)part * blockDim.x + threadIdx.x; e < n; e += (long long)parts * blockDim.x) {
        const long long r = e / per;
        const int t = (int)(r / heads), h = (int)(r % heads), c = (int)(e % per);
        T* dst = static_cast<T*>(X) + (t < lo ? t : t - lo + hi) * s.tok + h * s.head + c * (16 / (int)sizeof(T));
        *reinterpret_cast<uint4*>(dst) = make_uint4(0u, 0u, 0u, 0u);
    }
}

template <typename T>
__device__ void fill_grads(const PackedBwd& a, bool all, int part, int parts) {
    const int q_lo = all ? 0 : a.cu_q[0], q_hi = all ? 0 : a.cu_q[a.N];
    const int k_lo = all ? 0 : a.cu_k[0], k_hi = all ? 0 : a.cu_k[a.N];
    zero_rows<T>(a.dQ, a.sdq, a.H, a.d, q_lo, q_hi, a.T_q, part, parts);
    zero_rows<T>(a.dK, a.sdk, a.H_kv, a.d, k_lo, k_hi, a.T_k, part, parts);
    zero_rows<T>(a.dV, a.sdv, a.H_kv, a.d, k_lo, k_hi, a.T_k, part, parts);
}

constexpr int kBuckets = 2048;
constexpr int kBwdSmemSeqs = 2047;  // sequences whose tile offsets are kept in shared memory
constexpr int kSmallPlan = 256;     // threads of a plan block that has no more of anything to place

// Block 0 plans; blocks 1 .. map_blocks write tensor maps, one warp a map; the rest fill.
__global__ void __launch_bounds__(kPlanThreads, 1)
    bwd_plan_kernel(const PackedBwd a, const BwdPlan p, const __grid_constant__ BwdMaps maps, int map_blocks) {
    ptx::griddep_launch_dependents();
    const int tid = threadIdx.x;
    if ((int)blockIdx.x > map_blocks) {
        const int part = blockIdx.x - 1 - map_blocks, parts = gridDim.x - 1 - map_blocks;
        const bool all = any_bad(a);  // nothing is computed then: no row is left unset
        if (a.dtype == FA_F32)
            fill_grads<float>(a, all, part, parts);
        else
            fill_grads<__half>(a, all, part, parts);
        return;
    }
    if (blockIdx.x > 0) {
        __shared__ __align__(128) uint32_t s_map[kPlanThreads / 32][32];
        const int lane = tid & 31, w = tid >> 5;
        const long long i = (long long)(blockIdx.x - 1) * (blockDim.x / 32) + w;
        const int n = (int)(i / kSeqMaps), which = (int)(i % kSeqMaps);
        if (n >= a.N || (which == 4 && a.d == 256)) return;  // that kernel adds without a map
        Seq s;
        seq_at(a, n, s);
        const bool q = which < 2 || which == 4;
        const int len = q ? s.nq : s.nk;
        if (len == 0) return;  // never loaded
        const void* base = which == 0 ? a.Q : which == 1 ? a.dO : which == 2 ? a.K : which == 3 ? a.V : p.dqacc;
        // bytes from a row to the next
        const long long row = which == 4 ? (long long)a.H * a.d * 4
                                         : (which == 0 ? a.sq : which == 1 ? a.sdo : which == 2 ? a.sk : a.sv).tok * 2;
        write_map(p.maps + i, &maps.m[which], ptx::smem_u32(s_map[w]), s_map[w],
                  static_cast<const char*>(base) + (q ? s.q0 : s.k0) * row, len, lane);
        return;
    }
    __shared__ long long s_sum[33];
    __shared__ int s_count[kBuckets];
    __shared__ int s_first[2][kBwdSmemSeqs + 1];
    const int threads = blockDim.x;
    // first query and key tile of each sequence (in shared memory where they fit)
    int* first_q = a.N <= kBwdSmemSeqs ? s_first[0] : p.seq_q;
    int* first_k = a.N <= kBwdSmemSeqs ? s_first[1] : p.seq_k;
    long long tiles = 0;  // query tiles | key tiles << 32
    bool bad = false;
    for (int n0 = 0; n0 < a.N; n0 += threads) {
        const int n = n0 + tid;
        Seq s = {0, 0, 0, 0};
        if (n < a.N && !seq_at(a, n, s)) bad = true;
        long long total;
        const long long at = tiles + block_excl_scan((long long)((s.nq + kBwdTile - 1) / kBwdTile) |
                                                         (long long)((s.nk + kBwdTile - 1) / kBwdTile) << 32,
                                                     s_sum, &total);
        if (n < a.N) {
            first_q[n] = (int)at;
            first_k[n] = (int)(at >> 32);
            p.seq_q[n] = (int)at;
        }
        tiles += total;
    }
    int UQ = (int)tiles, UK = (int)(tiles >> 32);
    if (tid == 0) {
        first_q[a.N] = UQ;
        first_k[a.N] = UK;
        p.seq_q[a.N] = UQ;
        *p.ticket = 0u;
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) atomicOr(a.err, kErrLengths);
        UQ = UK = 0;
    }
    if (tid == 0) p.head[0] = UQ;
    if (a.deterministic)
        for (long long i = tid; i < (long long)a.H * p.max_units; i += threads) p.sem[i] = 0u;
    for (int u = tid; u < UQ; u += threads) {
        const int n = find_seq(first_q, a.N, u);
        const int i0 = (u - first_q[n]) * kBwdTile, q0 = a.cu_q[n], nq = a.cu_q[n + 1] - q0;
        p.query[u] = {q0 + i0, min(kBwdTile, nq - i0)};
    }
    long long its = 0;
    int mine = 0;  // query tiles of the thread's key tile in the first round
    for (int v = tid; v < UK; v += threads) {
        const int n = find_seq(first_k, a.N, v);
        Seq s;
        seq_at(a, n, s);
        KeyTile t;
        t.n = n;
        t.n0 = (v - first_k[n]) * kBwdTile;
        t.k_tok = s.k0 + t.n0;
        t.S_q = s.nq;
        t.S_k = s.nk;
        t.unit0 = first_q[n];
        Shape sh;
        sh.S_q = s.nq;
        sh.S_k = s.nk;
        sh.causal = a.causal;
        sh.window = a.window;
        int lo, hi;
        query_range(sh, t.n0, min(t.n0 + kBwdTile, s.nk), lo, hi);
        t.its = hi > lo ? (hi + kBwdTile - 1) / kBwdTile - lo / kBwdTile : 0;
        t.q_tok = s.q0;
        p.key[v] = t;
        if (v == tid) mine = t.its;
        its += t.its;
    }
    // iterations of an even share
    const int g = a.H / a.H_kv;
    long long all;
    block_excl_scan(its, s_sum, &all);
    const long long share = max((all * a.H + p.shares - 1) / p.shares, (long long)p.min_its);
    // iterations, and parts, of tile v
    auto length = [&](int v) { return v < UK ? (long long)(v == tid ? mine : p.key[v].its) * g : 0; };
    auto parts_of = [&](int v, long long n) { return v >= UK ? 0 : n > share ? (int)((n + share - 1) / share) : 1; };
    // Works in tile order, or sorted by length, most first, when they take more than one round of
    // CTAs.  Running totals: works | cut tiles << 32 | slots << 48 (both below 2 x 16 bits: the
    // cut tiles are fewer than the SMs).
    const bool in_order = a.deterministic || UK <= threads;
    bool sorted = !a.deterministic;
    if (!in_order) {
        for (int i = tid; i < kBuckets; i += threads) s_count[i] = 0;
        __syncthreads();
    }
    long long run = 0;
    for (int v0 = 0; v0 < UK; v0 += threads) {
        const int v = v0 + tid;
        const long long len = length(v);
        const int n = parts_of(v, len);
        long long total;
        const long long at =
            run + block_excl_scan((long long)n | (n > 1 ? 1ll << 32 | (long long)n << 48 : 0ll), s_sum, &total);
        const int w = (int)at, slot = (int)(at >> 48);
        if (n > 1) p.cut[(int)(at >> 32) & 0xffff] = {v, 0, n, slot};
        run += total;
        if (in_order) {
            // one round of CTAs: their order does not matter
            if (UK <= threads && (long long)(int)run * a.H_kv <= p.one_round) sorted = false;
            if (!sorted)
                for (int i = 0; i < n; ++i) p.work[w + i] = {v, i, n, slot + i};
        } else if (n > 0) {
            atomicAdd(&s_count[(int)min((len + n - 1) / n, (long long)kBuckets - 1)], n);
        }
    }
    if (tid == 0) {
        p.head[1] = (int)run;
        p.head[2] = (int)(run >> 32) & 0xffff;
    }
    if (!sorted) return;
    if (in_order) {  // one round of tiles, more than one of CTAs: count them now
        for (int i = tid; i < kBuckets; i += threads) s_count[i] = 0;
        __syncthreads();
        const long long len = length(tid);
        const int n = parts_of(tid, len);
        if (n > 0) atomicAdd(&s_count[(int)min((len + n - 1) / n, (long long)kBuckets - 1)], n);
    }
    __syncthreads();
    // first place of each bucket, longest first (within a bucket in any order)
    const int per = kBuckets / threads;
    long long sum = 0, total;
    for (int i = 0; i < per; ++i) sum += s_count[kBuckets - 1 - (tid * per + i)];
    int at = (int)block_excl_scan(sum, s_sum, &total);
    for (int i = 0; i < per; ++i) {
        int& c = s_count[kBuckets - 1 - (tid * per + i)];
        const int n = c;
        c = at;
        at += n;
    }
    __syncthreads();
    run = 0;
    for (int v0 = 0; v0 < UK; v0 += threads) {
        const int v = v0 + tid;
        const long long len = length(v);
        const int n = parts_of(v, len);
        const long long slot = run + block_excl_scan(n > 1 ? (long long)n : 0ll, s_sum, &total);
        run += total;
        const int w = n > 0 ? atomicAdd(&s_count[(int)min((len + n - 1) / n, (long long)kBuckets - 1)], n) : 0;
        for (int i = 0; i < n; ++i) p.work[w + i] = {v, i, n, (int)slot + i};
    }
}

bool row_map(CUtensorMap* m, const void* base, CUtensorMapDataType dt, int es, int d, int heads, long long rows,
             long long head_stride, long long row_stride, int box_rows) {
    TmaEncodeTiledFn enc = tma_encode_fn();
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t str[2] = {(cuuint64_t)head_stride * es, (cuuint64_t)row_stride * es};
    const cuuint32_t box[3] = {(cuuint32_t)(128 / es), 1, (cuuint32_t)box_rows};
    const cuuint32_t one[3] = {1, 1, 1};
    return enc && enc(m, dt, 3, const_cast<void*>(base), dims, str, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_bwd_plan(const PackedBwd& a, const BwdPlan& p, bool tensor_cores, cudaStream_t st) {
    static_assert(kBuckets % kPlanThreads == 0 && kBuckets % kSmallPlan == 0, "whole buckets a thread");
    const bool small = a.N <= kSmallPlan && p.max_units <= kSmallPlan && p.max_keys <= kSmallPlan;
    const int threads = small ? kSmallPlan : kPlanThreads;
    BwdMaps maps = {};
    int map_blocks = 0;
    if (tensor_cores) {
        const CUtensorMapDataType dt =
            a.dtype == FA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
        const int rows = a.d == 256 ? 64 : kBwdTile;  // of the kernel's tiles
        // an empty axis is never loaded: its maps are built over the other axis' rows
        const void* q = a.T_q > 0 ? a.Q : a.K;
        const void* g = a.T_q > 0 ? a.dO : a.K;
        const void* k = a.T_k > 0 ? a.K : a.Q;
        const void* v = a.T_k > 0 ? a.V : a.Q;
        if (!row_map(&maps.m[0], q, dt, 2, a.d, a.H, 1, a.sq.head, a.sq.tok, rows) ||
            !row_map(&maps.m[1], g, dt, 2, a.d, a.H, 1, a.sdo.head, a.sdo.tok, rows) ||
            !row_map(&maps.m[2], k, dt, 2, a.d, a.H_kv, 1, a.sk.head, a.sk.tok, rows) ||
            !row_map(&maps.m[3], v, dt, 2, a.d, a.H_kv, 1, a.sv.head, a.sv.tok, rows))
            return cudaErrorInvalidValue;
        // the accumulator: boxes of 32 fp32 columns
        if (a.d <= 128 && !row_map(&maps.m[4], p.dqacc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, a.d, a.H, 1, a.d,
                                   (long long)a.H * a.d, kBwdTile))
            return cudaErrorInvalidValue;
        map_blocks = (int)(((long long)a.N * kSeqMaps + threads / 32 - 1) / (threads / 32));
    }
    bwd_plan_kernel<<<1 + map_blocks + (a.fill ? 32 : 0), threads, 0, st>>>(a, p, maps, map_blocks);
    return cudaGetLastError();
}

cudaError_t launch_fwd_plan(const PackedFwd& a, const FwdGeom& g, const FwdPlan& p, cudaStream_t st) {
    fwd_plan_kernel<<<a.fill ? 33 : 1, kPlanThreads, 0, st>>>(a, g, p);
    return cudaGetLastError();
}

}  // namespace fa
