// packed.cuh -- shared definitions of the packed and paged attention operators (not part of
// the C ABI): call arguments, the work plan that a small kernel builds on the device from the
// sequence lengths, and how a CTA walks its share of it.
//
// Packed tensors are token major: Q [T_q, H, d], K and V [T_k, H_kv, d]; sequence n owns query
// rows [cu_q[n], cu_q[n+1]) and key rows [cu_k[n], cu_k[n+1]).  Paged calls take K and V from a
// cache [pages, page_size, H_kv, d]: key j of request n is row j % page_size of page
// table[n][j / page_size], and the request holds seq_lens[n] keys.  Inside a sequence query i
// sits at key position i + S_k - S_q, as in the dense calls.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "fa_internal.cuh"
#include "sm103_ptx.cuh"

namespace fa {

struct RowStride {
    long long tok, head;  // elements
};

// One forward call (packed: cu_k set; paged: seq_lens and table set).
struct PackedFwd {
    const void *Q, *K, *V;
    void* O;
    float* LSE;  // [H, T_q]
    const int *cu_q, *cu_k, *seq_lens, *table;
    int N, T_q, T_k, H, H_kv, d;
    int pages, page_size, max_pages;
    RowStride q, k, v, o;
    long long k_page, v_page;  // elements from one page to the next
    float scale;
    int causal, window, fill, dtype;
    unsigned int* err;
    bool paged() const { return cu_k == nullptr; }
};

// ---------------------------------------------------------------- forward plan
// A unit is `tpt` consecutive query tokens of one sequence; the g query heads of a key/value
// head are packed beside each other, so a tile has tpt * g rows (token major, then head) and
// reads each key once for the whole group.  A (unit, head) item takes `overhead` positions for
// what it costs beside its key tiles (the epilogue), then one per key tile (one if it has none).
// The plan lays the items out on one axis of W positions and gives every CTA the same number of
// consecutive ones, so the grid is filled whatever the lengths are.  A tile belongs to the CTA
// that has its position; an item whose tiles belong to several CTAs is computed in parts and
// joined by the last of them to finish.
struct alignas(16) FwdTile {
    int n;        // sequence
    int q_tok;    // first query token (row of Q)
    int n_tok;    // query tokens of the unit
    int pos0;     // key position of the first token
    int k_base;   // packed: first key row of the sequence
    int S_k;      // keys of the sequence (paged: of those the table has room for)
    int n_first;  // first key tile that a row sees
    int n_cnt;    // key tiles [n_first, n_first + n_cnt) hold every key a row sees
};
static_assert(sizeof(FwdTile) == 32, "loaded as two 16-byte words");

struct FwdPlan {
    FwdTile* tile;    // [units]
    long long* base;  // [units] first position of the unit
    long long* head;  // [0] W, [1] positions per CTA
    int* start;       // [ctas] unit that holds the CTA's first position
    int* seq_units;   // [N + 1] first unit of each sequence
    // [ctas] parts finished of the item whose first tile is the CTA's: (tag << 16) | count.  A
    // word with another tag counts as zero and the last part leaves zero, so the workspace needs
    // no clearing and a replayed call (which has its tag again) starts clean.
    unsigned long long* done;
    unsigned long long tag;  // of this call, 48 bits, never 0
    // parts of cut items, two per CTA (2c: continues an item, 2c + 1: starts one): fp32
    // accumulators, not divided by the row sum, and (running max in log2 units, row sum)
    float* part_o;    // [2 ctas][rows][D]
    float2* part_ml;  // [2 ctas][rows]
};

// Tile shape a forward kernel asks the plan for.
struct FwdGeom {
    int rows;       // rows of a tile
    int tpt;        // query tokens per unit
    int bn;         // keys per tile
    int heads;      // items per unit
    int ctas;       // CTAs of the grid
    int D;          // columns of a part
    int min_chunk;  // positions per CTA at least
    int overhead;   // positions an item takes beside its key tiles
    bool self;      // every CTA plans for itself (few units): no plan kernel, tiles per CTA
};
constexpr int kSelfUnits = 896;  // units (and sequences) a CTA plans for itself at most

inline size_t packed_align(size_t x) { return (x + 255) / 256 * 256; }
inline long long plan_units(const PackedFwd& a, const FwdGeom& g) {
    return a.T_q / g.tpt + (a.N < a.T_q ? a.N : a.T_q) + 1;
}
// A tag no earlier call of the process had.
unsigned long long next_tag();
// Lays the plan out in `ws`; returns the bytes it needs.
inline size_t fwd_plan_layout(const PackedFwd& a, const FwdGeom& g, void* ws, FwdPlan* p) {
    char* b = static_cast<char*>(ws);
    const size_t U = (size_t)plan_units(a, g), C = (size_t)g.ctas;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char* r = b + at;
        at = packed_align(at + bytes);
        return r;
    };
    FwdPlan q;
    q.head = reinterpret_cast<long long*>(take(16));
    q.tile = reinterpret_cast<FwdTile*>(take((g.self ? C : 1) * U * sizeof(FwdTile)));
    q.base = reinterpret_cast<long long*>(take(U * 8));
    q.start = reinterpret_cast<int*>(take(C * 4));
    q.done = reinterpret_cast<unsigned long long*>(take(C * 8));
    q.tag = 0;
    q.seq_units = reinterpret_cast<int*>(take(((size_t)a.N + 1) * 4));
    q.part_ml = reinterpret_cast<float2*>(take(2 * C * g.rows * 8));
    q.part_o = reinterpret_cast<float*>(take(2 * C * g.rows * g.D * 4));
    if (p) *p = q;
    return at;
}

// Counts a part of an item in; true for the last of `count`.
__device__ __forceinline__ bool arrive_part(unsigned long long* word, unsigned long long tag, int count) {
    unsigned long long seen = *reinterpret_cast<volatile unsigned long long*>(word);
    while (true) {
        const int n = (seen >> 16) == tag ? (int)(seen & 0xffff) : 0;
        const unsigned long long next = n + 1 == count ? 0ull : (tag << 16) | (unsigned)(n + 1);
        const unsigned long long old = atomicCAS(word, seen, next);
        if (old == seen) return n + 1 == count;
        seen = old;
    }
}

// Where a CTA starts.
struct FwdShare {
    const FwdTile* tile;       // by unit
    long long W, chunk, base;  // positions in all and per CTA; first position of unit u
    int u;
    __device__ __forceinline__ void read(const FwdPlan& p, int cta) {
        tile = p.tile;
        W = p.head[0];
        chunk = p.head[1];
        u = chunk * cta < W ? p.start[cta] : 0;
        base = chunk * cta < W ? p.base[u] : 0;
    }
};

// A CTA's walk over its positions: segments (unit, head, key tiles [j0, j1)).
struct FwdWalk {
    long long item, start, end, chunk;  // first position of the item's tiles; the CTA's positions
    int u, hd, j0, j1, cc, heads, overhead;
    FwdTile t;
    const FwdTile* tile;
    __device__ __forceinline__ void load() {
        const int4* r = reinterpret_cast<const int4*>(tile + u);
        const int4 a = r[0], b = r[1];
        t.n = a.x, t.q_tok = a.y, t.n_tok = a.z, t.pos0 = a.w;
        t.k_base = b.x, t.S_k = b.y, t.n_first = b.z, t.n_cnt = b.w;
        cc = t.n_cnt > 0 ? t.n_cnt : 1;
    }
    // tiles of the item that belong to the CTA; false if there are none
    __device__ __forceinline__ bool cut() {
        if (item >= end) return false;
        j0 = start > item ? (int)(start - item) : 0;
        j1 = end - item < cc ? (int)(end - item) : cc;
        return true;
    }
    __device__ __forceinline__ bool init(const FwdShare& s, int cta, int heads_, int overhead_) {
        heads = heads_;
        overhead = overhead_;
        chunk = s.chunk;
        start = chunk * cta;
        end = start + chunk < s.W ? start + chunk : s.W;
        if (start >= end) return false;
        tile = s.tile;
        u = s.u;
        load();
        hd = (int)((start - s.base) / (cc + overhead));
        item = s.base + (long long)hd * (cc + overhead) + overhead;
        return cut();
    }
    __device__ __forceinline__ bool next() {
        item += cc;
        if (item >= end) return false;  // the next item's first position
        if (++hd == heads) {
            hd = 0;
            ++u;
            load();
        }
        item += overhead;
        return cut();
    }
    __device__ __forceinline__ int tiles() const { return t.n_cnt > 0 ? j1 - j0 : 0; }
    __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == cc; }
    // of a cut item: the CTA its first tile belongs to, and its number of parts
    __device__ __forceinline__ void parts(int& first, int& count) const {
        first = (int)(item / chunk);
        count = (int)((item + cc - 1) / chunk) - first + 1;
    }
};

// ---------------------------------------------------------------- planning, device side
// (here for the plan kernels and for the CTAs that plan for themselves)
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

// Exclusive scan over the block; *total gets the block's sum.  sums: 33 values.  Ends with a barrier.
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

// Keys that a request's row of the table has room for.
__device__ __forceinline__ long long table_room(const PackedFwd& a) { return (long long)a.max_pages * a.page_size; }

// Lengths of sequence n; false (and empty) if they do not fit the tensors.  A request may be longer
// than its row of the table: the keys behind it are not in the cache and not seen (make_tile).
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
        const bool okk = nk >= 0 && nk <= (1 << 28);  // what positions are kept for
        s.k0 = 0;
        s.nk = okk ? nk : 0;
        ok = ok && okk;
    }
    return ok;
}

// Whether a request with new tokens is longer than its row of the table; to be reported.
__device__ __forceinline__ bool past_table(const PackedFwd& a, const Seq& s) {
    return a.cu_k == nullptr && s.nq > 0 && s.nk > table_room(a);
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

// Unit `i` of sequence n; its positions per head.
__device__ __forceinline__ int make_tile(const PackedFwd& a, const FwdGeom& g, int n, int i, FwdTile& t) {
    Seq s;
    seq_at(a, n, s);
    const int i0 = i * g.tpt;
    t.n = n;
    t.q_tok = s.q0 + i0;
    t.n_tok = min(g.tpt, s.nq - i0);
    t.pos0 = i0 + s.nk - s.nq;
    t.k_base = s.k0;
    t.S_k = a.cu_k == nullptr ? (int)min((long long)s.nk, table_room(a)) : s.nk;
    Shape sh;
    sh.S_q = s.nq;
    sh.S_k = s.nk;
    sh.causal = a.causal;
    sh.window = a.window;
    int lo, hi;
    key_range(sh, i0, i0 + t.n_tok, lo, hi);
    hi = min(hi, t.S_k);
    t.n_first = hi > lo ? lo / g.bn : 0;
    t.n_cnt = hi > lo ? (hi + g.bn - 1) / g.bn - t.n_first : 0;
    return max(t.n_cnt, 1) + g.overhead;
}

__device__ __forceinline__ long long share_of(long long W, const FwdGeom& g) {
    const long long c = (W + g.ctas - 1) / g.ctas;
    return c < g.min_chunk ? g.min_chunk : c;
}

// Rows before the first and behind the last sequence, or (all) every row: O = 0, LSE = -inf.
template <typename T>
__device__ __forceinline__ void fill_rows(const PackedFwd& a, bool all, long long first, long long step) {
    const int lo = all ? 0 : a.cu_q[0], hi = all ? 0 : a.cu_q[a.N];
    const int per = a.d * (int)sizeof(T) / 16;
    const long long n = (long long)(lo + a.T_q - hi) * a.H * per;
    for (long long e = first; e < n; e += step) {
        const long long r = e / per;
        const int t = (int)(r / a.H), h = (int)(r % a.H), c = (int)(e % per);
        const int tok = t < lo ? t : t - lo + hi;
        T* dst = static_cast<T*>(a.O) + tok * a.o.tok + h * a.o.head + c * (16 / (int)sizeof(T));
        *reinterpret_cast<uint4*>(dst) = make_uint4(0u, 0u, 0u, 0u);
        if (c == 0) a.LSE[(size_t)h * a.T_q + tok] = -INFINITY;
    }
}

// Scratch of plan_self in shared memory.
struct SelfPlan {
    long long lsum[33];
    FwdShare share;
    int isum[33];
    int first[kSelfUnits + 1];
};

// The plan kernel's work, done by every CTA (kThreads threads) for itself: the same plan, of
// which it keeps the units that hold its positions.  Reads a few KB of lengths; saves a launch.
template <int kThreads>
__device__ __forceinline__ void plan_self(const PackedFwd& a, const FwdGeom& g, const FwdPlan& p, int max_units,
                                          SelfPlan* s) {
    const int tid = threadIdx.x, cta = blockIdx.x;
    bool bad = false;
    int U = 0;
    for (int n0 = 0; n0 < a.N; n0 += kThreads) {
        const int n = n0 + tid;
        Seq q = {0, 0, 0, 0};
        if (n < a.N && !seq_at(a, n, q)) bad = true;
        if (past_table(a, q) && cta == 0) atomicOr(a.err, kErrLengths);
        int total;
        const int at = block_excl_scan((q.nq + g.tpt - 1) / g.tpt, s->isum, &total);
        if (n < a.N) s->first[n] = U + at;
        U += total;
    }
    if (tid == 0) s->first[a.N] = U;
    if (__syncthreads_or(bad)) {  // lengths that do not fit the tensors: nothing is computed
        if (tid == 0 && cta == 0) atomicOr(a.err, kErrLengths);
        U = 0;
    }
    constexpr int kRounds = (kSelfUnits + kThreads - 1) / kThreads;
    FwdTile t[kRounds];
    int cost[kRounds];  // per head
    long long base[kRounds], W = 0;
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
        const int u = i * kThreads + tid;
        cost[i] = 0;
        if (i * kThreads >= U) continue;
        if (u < U) {
            const int n = find_seq(s->first, a.N, u);
            cost[i] = make_tile(a, g, n, u - s->first[n], t[i]);
        }
        long long total;
        base[i] = W + block_excl_scan((long long)cost[i] * g.heads, s->lsum, &total);
        W += total;
    }
    const long long chunk = share_of(W, g);
    const long long lo = chunk * cta, hi = lo + chunk;
    FwdTile* mine = p.tile + (size_t)cta * max_units;
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
        const int u = i * kThreads + tid;
        if (u >= U) continue;
        const long long end = base[i] + (long long)cost[i] * g.heads;
        if (base[i] < hi && end > lo) mine[u] = t[i];
        if (base[i] <= lo && end > lo) {
            s->share.u = u;
            s->share.base = base[i];
        }
    }
    if (tid == 0) {
        s->share.tile = mine;
        s->share.W = W;
        s->share.chunk = chunk;
    }
    __syncthreads();
}

// From a row's running max m (log2 units) and sum l.  l is 0 only for a row that sees no key (or
// none with a score above -inf): O = 0, LSE = -inf.  A NaN sum stays NaN in both.
__device__ __forceinline__ float inv_sum(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}
// The max of a part with the sum's NaN: the max itself leaves NaN out (-inf where all scores are NaN).
__device__ __forceinline__ float part_max(float m, float l) { return isnan(l) ? l : m; }

// packed_plan.cu
cudaError_t launch_fwd_plan(const PackedFwd& a, const FwdGeom& g, const FwdPlan& p, cudaStream_t st);

// Joins the parts of one cut item (kThreads threads, all of them past the barrier that follows
// the last part's arrival): O = sum_k O_k 2^(m_k - M) / sum_k l_k 2^(m_k - M), parts in the order
// of their keys.  m_k = -inf is a row that sees no key in a part, m_k = NaN one whose scores there hold
// a NaN (part_max), which reaches the result.
// s_row: `rows` float2 of shared memory; sync: a barrier of those threads.
template <typename T, int kThreads, int kRowsLd, int kD, int kBatch, typename Sync>
__device__ __forceinline__ void join_parts(const PackedFwd& a, const FwdPlan& p, const FwdTile& t, int head0, int g,
                                           int rows, int first, int count, int tid, float2* s_row, Sync sync) {
    auto slot = [&](int k) { return (size_t)(k == 0 ? 2 * first + 1 : 2 * (first + k)) * kRowsLd; };
    for (int r = tid; r < rows; r += kThreads) {
        float M = -INFINITY, L = 0.f;
#pragma unroll 4
        for (int k = 0; k < count; ++k) {
            const float2 ml = __ldcg(&p.part_ml[slot(k) + r]);
            if (ml.x > M) {
                L = L * exp2f(M - ml.x) + ml.y;
                M = ml.x;
            } else if (ml.x != -INFINITY) {
                L += ml.y * exp2f(ml.x - M);
            }
        }
        s_row[r] = make_float2(M, inv_sum(L));
        a.LSE[(size_t)(head0 + r % g) * a.T_q + t.q_tok + r / g] = lse_of(M, L);
    }
    sync();
    // four columns of a row per thread and step; kBatch steps' loads in flight together
    constexpr int C4 = kD / 4;
    for (int e0 = tid; e0 < rows * C4; e0 += kBatch * kThreads) {
        float4 s[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) s[b] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < count; ++k) {
            float4 o[kBatch];
            float w[kBatch];
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int e = e0 + b * kThreads, r = e / C4;
                if (r < rows) {
                    o[b] = __ldcg(reinterpret_cast<const float4*>(p.part_o + (slot(k) + r) * kD) + e % C4);
                    w[b] = __ldcg(&p.part_ml[slot(k) + r]).x;
                }
            }
#pragma unroll
            for (int b = 0; b < kBatch; ++b) {
                const int r = (e0 + b * kThreads) / C4;
                // a part in which the row sees no key adds nothing
                if (r < rows && w[b] != -INFINITY) {
                    const float f = exp2f(w[b] - s_row[r].x);
                    s[b].x += o[b].x * f, s[b].y += o[b].y * f, s[b].z += o[b].z * f, s[b].w += o[b].w * f;
                }
            }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int e = e0 + b * kThreads, r = e / C4, c = e % C4 * 4;
            if (r >= rows || c >= a.d) continue;
            const float inv = s_row[r].y;
            T* dst = static_cast<T*>(a.O) + (t.q_tok + r / g) * a.o.tok + (head0 + r % g) * a.o.head + c;
            alignas(16) T out[4] = {TypeTraits<T>::from_f32(s[b].x * inv), TypeTraits<T>::from_f32(s[b].y * inv),
                                    TypeTraits<T>::from_f32(s[b].z * inv), TypeTraits<T>::from_f32(s[b].w * inv)};
            if constexpr (sizeof(T) == 4)
                *reinterpret_cast<float4*>(dst) = *reinterpret_cast<const float4*>(out);
            else
                *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(out);
        }
    }
}

// Raises a kernel's shared-memory limit once per device; `ready` has a bit per device.
template <typename K>
inline cudaError_t allow_smem(K* kern, int bytes, std::atomic<uint64_t>& ready) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (ready.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_release);
    return e;
}

// Forward launchers: with ws == nullptr only *bytes (the workspace they need) is set.
// packed_fwd.cu: tensor cores (f16 / bf16)
cudaError_t launch_packed_fwd(const PackedFwd& a, void* ws, size_t* bytes, cudaStream_t st);
// packed_simt.cu: CUDA cores (f32, and layouts that TMA cannot address)
cudaError_t launch_packed_fwd_simt(const PackedFwd& a, void* ws, size_t* bytes, cudaStream_t st);

// ---------------------------------------------------------------- backward
struct PackedBwd {
    const void *dO, *Q, *K, *V, *O;
    const float* LSE;  // [H, T_q]
    void *dQ, *dK, *dV;
    const int *cu_q, *cu_k;
    int N, T_q, T_k, H, H_kv, d;
    RowStride sdo, sq, sk, sv, so, sdq, sdk, sdv;
    float scale;
    int causal, window, deterministic, fill, dtype;
    unsigned int* err;
};

constexpr int kBwdTile = 128;  // query rows and key rows of a plan tile
constexpr int kSeqMaps = 5;    // tensor maps of a sequence

// A 128-row query tile: rows q_tok .. q_tok + rows - 1 of Q and of the accumulator; its place in the
// list is its place in the padded rows of D and the LSE copy.
struct QueryTile {
    int q_tok, rows;
};
// A 128-row key tile of a sequence.
struct alignas(16) KeyTile {
    int n;      // sequence
    int k_tok;  // first key row of the tile (row of K)
    int n0;     // the same within the sequence
    int S_q, S_k;
    int unit0;  // first query tile of the sequence
    int its;    // query tiles that see a key of this tile
    int q_tok;  // first query row of the sequence (row of Q)
};
// What one CTA does of a key tile (for one key/value head): share `part` of `parts` of its
// (query tile, query head) iterations.  A tile with more iterations than an even share of the
// whole call over the SMs is cut: its parts leave fp32 sums of dK and dV in slots `slot` on,
// which the pass after the main kernel adds up in order.
struct alignas(16) KeyWork {
    int tile, part, parts, slot;
};

struct BwdPlan {
    long long* head;      // [0] query tiles, [1] works, [2] cut key tiles
    QueryTile* query;     // [max_units]
    KeyTile* key;         // [max_keys], in sequence order
    KeyWork* work;        // [max_work], longest first (deterministic: in order of the tiles)
    KeyWork* cut;         // [max_cut] tiles with more than one part (slot: the first part's)
    float* part;          // [max_slots][H_kv][2: dV, dK][128][d] fp32 sums of the parts
    int *seq_q, *seq_k;   // [N + 1] first query / key tile of each sequence
    CUtensorMap* maps;    // [N][kSeqMaps] of each sequence: Q, dO, K, V, accumulator (tensor cores)
    unsigned *sem, *ticket;  // deterministic: turn counters [H][max_units], start-order ticket
    float *lse2, *D;      // [H][rows]
    float* dqacc;         // [T_q][H][d] fp32, not scaled
    long long rows;       // max_units * 128
    int max_units, max_keys, max_work, max_cut, max_slots;
    int shares;           // CTAs the iterations are spread over
    int one_round;        // CTAs of the main kernel (works x heads) that run at the same time
    int min_its;          // iterations a part has at least
};

int sm_count();  // of the current device (looked up once per device)

// CTAs that share the work of one plan tile and head, by their key rows.
inline int bwd_pieces(bool tensor_cores, int d) { return tensor_cores ? (d <= 128 ? 1 : 2) : (d <= 128 ? 2 : 4); }

inline size_t bwd_plan_layout(const PackedBwd& a, bool tensor_cores, void* ws, BwdPlan* p) {
    char* b = static_cast<char*>(ws);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        char* r = b + at;
        at = packed_align(at + bytes);
        return r;
    };
    BwdPlan q;
    q.max_units = a.T_q / kBwdTile + (a.N < a.T_q ? a.N : a.T_q);
    q.max_keys = a.T_k / kBwdTile + (a.N < a.T_k ? a.N : a.T_k);
    q.rows = (long long)q.max_units * kBwdTile;
    // with x = iterations / share of a tile, the tiles' x add up to shares / H_kv per head at
    // most, a cut tile has x > 1 and ceil(x) <= 2x parts.  On CUDA cores a plan tile is several
    // CTAs and a CTA's fixed cost is small: two rounds of CTAs even out better.
    const int pieces = bwd_pieces(tensor_cores, a.d);
    q.shares = ((tensor_cores ? 1 : 2) * sm_count() + pieces - 1) / pieces;
    q.one_round = sm_count() / pieces;
    q.min_its = 4;
    q.max_cut = q.shares / a.H_kv + 1;
    q.max_work = q.max_keys + q.max_cut;
    q.max_slots = 2 * q.max_cut;
    q.head = reinterpret_cast<long long*>(take(16));
    q.ticket = reinterpret_cast<unsigned*>(take(4));
    q.sem = reinterpret_cast<unsigned*>(take(a.deterministic ? (size_t)a.H * q.max_units * 4 : 0));
    q.query = reinterpret_cast<QueryTile*>(take((size_t)q.max_units * sizeof(QueryTile)));
    q.key = reinterpret_cast<KeyTile*>(take((size_t)q.max_keys * sizeof(KeyTile)));
    q.work = reinterpret_cast<KeyWork*>(take((size_t)q.max_work * sizeof(KeyWork)));
    q.cut = reinterpret_cast<KeyWork*>(take((size_t)q.max_cut * sizeof(KeyWork)));
    q.part = reinterpret_cast<float*>(take((size_t)q.max_slots * a.H_kv * 2 * kBwdTile * a.d * 4));
    q.seq_q = reinterpret_cast<int*>(take(((size_t)a.N + 1) * 4));
    q.seq_k = reinterpret_cast<int*>(take(((size_t)a.N + 1) * 4));
    q.maps = reinterpret_cast<CUtensorMap*>(take(tensor_cores ? (size_t)a.N * kSeqMaps * sizeof(CUtensorMap) : 0));
    q.lse2 = reinterpret_cast<float*>(take((size_t)q.rows * a.H * 4));
    q.D = reinterpret_cast<float*>(take((size_t)q.rows * a.H * 4));
    q.dqacc = reinterpret_cast<float*>(take((size_t)a.T_q * a.H * a.d * 4));
    if (p) *p = q;
    return at;
}

// packed_plan.cu: tiles, order, maps, counters; with a.fill the gradient rows of no sequence
cudaError_t launch_bwd_plan(const PackedBwd& a, const BwdPlan& p, bool tensor_cores, cudaStream_t st);
// packed_bwd_simt.cu: D, the LSE copy and a zeroed accumulator; dQ from the accumulator
cudaError_t launch_packed_preprocess(const PackedBwd& a, const BwdPlan& p, cudaStream_t st);
cudaError_t launch_packed_dq(const PackedBwd& a, const BwdPlan& p, cudaStream_t st);
// f16 / bf16: packed_bwd.cu (head dim <= 128), packed_bwd_d256.cu; f32: packed_bwd_simt.cu
cudaError_t launch_packed_bwd(const PackedBwd& a, const BwdPlan& p, cudaStream_t st);
cudaError_t launch_packed_bwd_d256(const PackedBwd& a, const BwdPlan& p, cudaStream_t st);
cudaError_t launch_packed_bwd_simt(const PackedBwd& a, const BwdPlan& p, cudaStream_t st);
// packed_bwd_simt.cu: the accumulator in deterministic mode where the main kernel leaves it out
// (f32, head dim 256)
cudaError_t launch_packed_dq_ordered(const PackedBwd& a, const BwdPlan& p, cudaStream_t st);

// Orders this thread's later uses of a tensor map after its writes (by an earlier kernel).
__device__ __forceinline__ void tensormap_acquire(const CUtensorMap* m) {
    asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// packed_api.cu: reads the error word of the packed and paged calls on the current device into
// *word and clears it, so that no bit set meanwhile is lost.  Returns an fa_status.
int packed_take_error_word(unsigned int* word);

// ---------------------------------------------------------------- page lookup
// The table's entry for key j of a request (-1 behind the table's last column) ...
__host__ __device__ __forceinline__ int page_entry(const int* row, int j, int page_size, int max_pages) {
    const int e = j / page_size;
    return e < max_pages ? row[e] : -1;
}
// ... and the page it names, or `pages` (one past the cache, which TMA reads as zeros and the
// CUDA-core kernel skips) with *bad set when the entry is not a page.
__host__ __device__ __forceinline__ int page_checked(int id, int pages, bool* bad) {
    if (id >= 0 && id < pages) return id;
    *bad = true;
    return pages;
}
__host__ __device__ __forceinline__ int page_of(const int* row, int j, int page_size, int max_pages, int pages,
                                                bool* bad) {
    return page_checked(page_entry(row, j, page_size, max_pages), pages, bad);
}

}  // namespace fa
