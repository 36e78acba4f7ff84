// packed_plan.cu -- work plans of the packed and paged operators, built on the device from the
// sequence lengths so that no call has to read them back.  One block plans (prefix sums over
// sequences and units, a few microseconds); the other blocks fill the output rows that belong
// to no sequence when the caller asked for that.
#include "packed.cuh"
#include "tma_map.cuh"

namespace fa {
namespace {

constexpr int kPlanThreads = 1024;

constexpr int kSmemSeqs = 4096;  // sequences whose unit offsets are also kept in shared memory

__global__ void __launch_bounds__(kPlanThreads, 1) fwd_plan_kernel(const PackedFwd a, const FwdGeom g, const FwdPlan p) {
    ptx::griddep_launch_dependents();
    if (blockIdx.x > 0) {
        const long long first = (long long)(blockIdx.x - 1) * blockDim.x + threadIdx.x;
        const long long step = (long long)(gridDim.x - 1) * blockDim.x;
        if (a.dtype == FA_F32)
            fill_rows<float>(a, first, step);
        else
            fill_rows<__half>(a, first, step);
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
    CUtensorMap m[4];  // Q, dO, K, V of the whole call
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
    if (lo < 0 || hi < lo || hi > T_all) return;  // reported by the planning block
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
__device__ void fill_grads(const PackedBwd& a, int part, int parts) {
    zero_rows<T>(a.dQ, a.sdq, a.H, a.d, a.cu_q[0], a.cu_q[a.N], a.T_q, part, parts);
    zero_rows<T>(a.dK, a.sdk, a.H_kv, a.d, a.cu_k[0], a.cu_k[a.N], a.T_k, part, parts);
    zero_rows<T>(a.dV, a.sdv, a.H_kv, a.d, a.cu_k[0], a.cu_k[a.N], a.T_k, part, parts);
}

__device__ __forceinline__ bool seq_at(const PackedBwd& a, int n, Seq& s) {
    const int q0 = a.cu_q[n], q1 = a.cu_q[n + 1], k0 = a.cu_k[n], k1 = a.cu_k[n + 1];
    const bool ok = q0 >= 0 && q1 >= q0 && q1 <= a.T_q && k0 >= 0 && k1 >= k0 && k1 <= a.T_k;
    s.q0 = q0;
    s.nq = ok ? q1 - q0 : 0;
    s.k0 = k0;
    s.nk = ok ? k1 - k0 : 0;
    return ok;
}

constexpr int kBuckets = 2048;

// Block 0 plans; blocks 1 .. map_blocks write tensor maps, one warp a map; the rest fill.
__global__ void __launch_bounds__(kPlanThreads, 1)
    bwd_plan_kernel(const PackedBwd a, const BwdPlan p, const __grid_constant__ BwdMaps maps, int map_blocks) {
    ptx::griddep_launch_dependents();
    const int tid = threadIdx.x;
    if ((int)blockIdx.x > map_blocks) {
        const int part = blockIdx.x - 1 - map_blocks, parts = gridDim.x - 1 - map_blocks;
        if (a.dtype == FA_F32)
            fill_grads<float>(a, part, parts);
        else
            fill_grads<__half>(a, part, parts);
        return;
    }
    if (blockIdx.x > 0) {
        __shared__ __align__(128) uint32_t s_map[kPlanThreads / 32][32];
        const int lane = tid & 31, w = tid >> 5;
        const long long i = (long long)(blockIdx.x - 1) * (kPlanThreads / 32) + w;
        const int n = (int)(i >> 2), which = (int)(i & 3);
        if (n >= a.N) return;
        Seq s;
        seq_at(a, n, s);
        const bool q = which < 2;
        const int len = q ? s.nq : s.nk;
        if (len == 0) return;  // never loaded
        const RowStride str = which == 0 ? a.sq : which == 1 ? a.sdo : which == 2 ? a.sk : a.sv;
        const void* base = which == 0 ? a.Q : which == 1 ? a.dO : which == 2 ? a.K : a.V;
        write_map(p.maps + i, &maps.m[which], ptx::smem_u32(s_map[w]), s_map[w],
                  static_cast<const char*>(base) + (long long)(q ? s.q0 : s.k0) * str.tok * 2, len, lane);
        return;
    }
    __shared__ int s_sum[33];
    __shared__ int s_count[kBuckets];
    // first query and key tile of each sequence
    int UQ = 0, UK = 0;
    bool bad = false;
    for (int n0 = 0; n0 < a.N; n0 += kPlanThreads) {
        const int n = n0 + tid;
        Seq s = {0, 0, 0, 0};
        if (n < a.N && !seq_at(a, n, s)) bad = true;
        int tq, tk;
        const int uq = block_excl_scan((s.nq + kBwdTile - 1) / kBwdTile, s_sum, &tq);
        const int uk = block_excl_scan((s.nk + kBwdTile - 1) / kBwdTile, s_sum, &tk);
        if (n < a.N) {
            p.seq_q[n] = UQ + uq;
            p.seq_k[n] = UK + uk;
        }
        UQ += tq;
        UK += tk;
    }
    if (tid == 0) {
        p.seq_q[a.N] = UQ;
        p.seq_k[a.N] = UK;
        if (p.ticket) *p.ticket = 0u;
    }
    if (__syncthreads_or(bad)) {
        if (tid == 0) atomicOr(a.err, kErrLengths);
        UQ = UK = 0;
    }
    if (tid == 0) p.head[0] = UQ;
    if (a.deterministic)
        for (long long i = tid; i < (long long)a.H * p.max_units; i += kPlanThreads) p.sem[i] = 0u;
    for (int i = tid; i < kBuckets; i += kPlanThreads) s_count[i] = 0;
    __syncthreads();
    for (int u = tid; u < UQ; u += kPlanThreads) {
        const int n = find_seq(p.seq_q, a.N, u);
        const int i0 = (u - p.seq_q[n]) * kBwdTile, q0 = a.cu_q[n], nq = a.cu_q[n + 1] - q0;
        p.query[u] = {q0 + i0, min(kBwdTile, nq - i0)};
    }
    long long its = 0;
    for (int v = tid; v < UK; v += kPlanThreads) {
        const int n = find_seq(p.seq_k, a.N, v);
        Seq s;
        seq_at(a, n, s);
        KeyTile t;
        t.n = n;
        t.n0 = (v - p.seq_k[n]) * kBwdTile;
        t.k_tok = s.k0 + t.n0;
        t.S_q = s.nq;
        t.S_k = s.nk;
        t.unit0 = p.seq_q[n];
        Shape sh;
        sh.S_q = s.nq;
        sh.S_k = s.nk;
        sh.causal = a.causal;
        sh.window = a.window;
        int lo, hi;
        query_range(sh, t.n0, min(t.n0 + kBwdTile, s.nk), lo, hi);
        t.its = hi > lo ? (hi + kBwdTile - 1) / kBwdTile - lo / kBwdTile : 0;
        t.pad = 0;
        p.key[v] = t;
        its += t.its;
    }
    // iterations of an even share
    const int g = a.H / a.H_kv;
    __shared__ long long s_lsum[33];
    long long all;
    block_excl_scan(its, s_lsum, &all);
    const long long share = max((all * a.H + p.shares - 1) / p.shares, (long long)p.min_its);
    // parts of each tile, in tile order; bucket sizes of the sort by length (most first)
    auto parts_of = [&](int v) {
        const long long n = v < UK ? (long long)p.key[v].its * g : 0;
        return v >= UK ? 0 : n > share ? (int)((n + share - 1) / share) : 1;
    };
    auto bucket = [&](int v, int parts) {
        return (int)min(((long long)p.key[v].its * g + parts - 1) / parts, (long long)kBuckets - 1);
    };
    int works = 0, cuts = 0, slots = 0;
    for (int v0 = 0; v0 < UK; v0 += kPlanThreads) {
        const int v = v0 + tid, n = parts_of(v);
        int total_w, total_c, total_s;
        const int w = works + block_excl_scan(n, s_sum, &total_w);
        const int c = cuts + block_excl_scan(n > 1 ? 1 : 0, s_sum, &total_c);
        const int sl = slots + block_excl_scan(n > 1 ? n : 0, s_sum, &total_s);
        if (n > 1) p.cut[c] = {v, 0, n, sl};
        if (a.deterministic)
            for (int i = 0; i < n; ++i) p.work[w + i] = {v, i, n, sl + i};
        else if (n > 0)
            atomicAdd(&s_count[bucket(v, n)], n);
        works += total_w;
        cuts += total_c;
        slots += total_s;
    }
    if (tid == 0) {
        p.head[1] = works;
        p.head[2] = cuts;
    }
    if (a.deterministic) return;
    __syncthreads();
    // counting sort, longest first (within a bucket in any order: it decides only which CTA
    // starts first)
    const int b0 = kBuckets - 1 - 2 * tid, b1 = b0 - 1;
    const int c0 = s_count[b0], c1 = s_count[b1];
    int total;
    const int at = block_excl_scan(c0 + c1, s_sum, &total);
    s_count[b0] = at;
    s_count[b1] = at + c0;
    __syncthreads();
    slots = 0;
    for (int v0 = 0; v0 < UK; v0 += kPlanThreads) {
        const int v = v0 + tid, n = parts_of(v);
        int total_s;
        const int sl = slots + block_excl_scan(n > 1 ? n : 0, s_sum, &total_s);
        const int w = n > 0 ? atomicAdd(&s_count[bucket(v, n)], n) : 0;
        for (int i = 0; i < n; ++i) p.work[w + i] = {v, i, n, sl + i};
        slots += total_s;
    }
}

bool row_map(CUtensorMap* m, const void* base, CUtensorMapDataType dt, int es, int d, int heads, long long rows,
             long long head_stride, long long row_stride) {
    TmaEncodeTiledFn enc = tma_encode_fn();
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t str[2] = {(cuuint64_t)head_stride * es, (cuuint64_t)row_stride * es};
    const cuuint32_t box[3] = {(cuuint32_t)(128 / es), 1, kBwdTile};
    const cuuint32_t one[3] = {1, 1, 1};
    return enc && enc(m, dt, 3, const_cast<void*>(base), dims, str, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool bwd_acc_map(CUtensorMap* m, const PackedBwd& a, const BwdPlan& p) {
    return row_map(m, p.dqacc, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, a.d, a.H, p.rows > 0 ? p.rows : 1, a.d,
                   (long long)a.H * a.d);
}

cudaError_t launch_bwd_plan(const PackedBwd& a, const BwdPlan& p, bool tensor_cores, cudaStream_t st) {
    static_assert(kBuckets == 2 * kPlanThreads, "two buckets a thread");
    BwdMaps maps = {};
    int map_blocks = 0;
    if (tensor_cores) {
        const CUtensorMapDataType dt =
            a.dtype == FA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
        // an empty axis is never loaded: its maps are built over the other axis' rows
        const void* q = a.T_q > 0 ? a.Q : a.K;
        const void* g = a.T_q > 0 ? a.dO : a.K;
        const void* k = a.T_k > 0 ? a.K : a.Q;
        const void* v = a.T_k > 0 ? a.V : a.Q;
        if (!row_map(&maps.m[0], q, dt, 2, a.d, a.H, 1, a.sq.head, a.sq.tok) ||
            !row_map(&maps.m[1], g, dt, 2, a.d, a.H, 1, a.sdo.head, a.sdo.tok) ||
            !row_map(&maps.m[2], k, dt, 2, a.d, a.H_kv, 1, a.sk.head, a.sk.tok) ||
            !row_map(&maps.m[3], v, dt, 2, a.d, a.H_kv, 1, a.sv.head, a.sv.tok))
            return cudaErrorInvalidValue;
        map_blocks = (int)(((long long)a.N * 4 + kPlanThreads / 32 - 1) / (kPlanThreads / 32));
    }
    bwd_plan_kernel<<<1 + map_blocks + (a.fill ? 32 : 0), kPlanThreads, 0, st>>>(a, p, maps, map_blocks);
    return cudaGetLastError();
}

cudaError_t launch_fwd_plan(const PackedFwd& a, const FwdGeom& g, const FwdPlan& p, cudaStream_t st) {
    fwd_plan_kernel<<<a.fill ? 33 : 1, kPlanThreads, 0, st>>>(a, g, p);
    return cudaGetLastError();
}

}  // namespace fa
