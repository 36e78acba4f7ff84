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
// reads each key once for the whole group.  A unit costs max(key tiles, 1) per head; the plan
// lays (unit, head, key tile) out on one axis of W positions and gives every CTA the same
// number of consecutive ones, so the grid is filled whatever the lengths are.  A (unit, head)
// item that a CTA boundary cuts is computed in parts and joined by the last CTA to finish.
struct alignas(16) FwdTile {
    int n;        // sequence
    int q_tok;    // first query token (row of Q)
    int n_tok;    // query tokens of the unit
    int pos0;     // key position of the first token
    int k_base;   // packed: first key row of the sequence
    int S_k;      // keys of the sequence
    int n_first;  // first key tile that a row sees
    int n_cnt;    // key tiles [n_first, n_first + n_cnt) hold every key a row sees
};
static_assert(sizeof(FwdTile) == 32, "loaded as two 16-byte words");

struct FwdPlan {
    FwdTile* tile;    // [units]
    long long* base;  // [units] first position of the unit
    long long* head;  // [0] W, [1] positions per CTA
    int* start;       // [ctas] unit that holds the CTA's first position
    unsigned* done;   // [ctas] parts finished of the item that starts in the CTA's range and leaves it
    int* seq_units;   // [N + 1] first unit of each sequence
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
};

inline size_t packed_align(size_t x) { return (x + 255) / 256 * 256; }
inline long long plan_units(const PackedFwd& a, const FwdGeom& g) {
    return a.T_q / g.tpt + (a.N < a.T_q ? a.N : a.T_q) + 1;
}
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
    q.tile = reinterpret_cast<FwdTile*>(take(U * sizeof(FwdTile)));
    q.base = reinterpret_cast<long long*>(take(U * 8));
    q.start = reinterpret_cast<int*>(take(C * 4));
    q.done = reinterpret_cast<unsigned*>(take(C * 4));
    q.seq_units = reinterpret_cast<int*>(take(((size_t)a.N + 1) * 4));
    q.part_ml = reinterpret_cast<float2*>(take(2 * C * g.rows * 8));
    q.part_o = reinterpret_cast<float*>(take(2 * C * g.rows * g.D * 4));
    if (p) *p = q;
    return at;
}

// A CTA's walk over its positions: segments (unit, head, key tiles [j0, j1)).
struct FwdWalk {
    long long pos, end, chunk, base;
    int u, hd, j0, j1, cc, heads;
    FwdTile t;
    __device__ __forceinline__ void load(const FwdPlan& p) {
        const int4* r = reinterpret_cast<const int4*>(p.tile + u);
        const int4 a = r[0], b = r[1];
        t.n = a.x, t.q_tok = a.y, t.n_tok = a.z, t.pos0 = a.w;
        t.k_base = b.x, t.S_k = b.y, t.n_first = b.z, t.n_cnt = b.w;
        cc = t.n_cnt > 0 ? t.n_cnt : 1;
    }
    __device__ __forceinline__ void cut() {
        const long long left = end - pos;
        j1 = left < cc - j0 ? j0 + (int)left : cc;
    }
    __device__ __forceinline__ bool init(const FwdPlan& p, int cta, int heads_) {
        heads = heads_;
        const long long W = p.head[0];
        chunk = p.head[1];
        pos = chunk * cta;
        end = pos + chunk < W ? pos + chunk : W;
        if (pos >= end) return false;
        u = p.start[cta];
        load(p);
        const long long rel = pos - p.base[u];
        hd = (int)(rel / cc);
        j0 = (int)(rel - (long long)hd * cc);
        cut();
        return true;
    }
    __device__ __forceinline__ bool next(const FwdPlan& p) {
        pos += j1 - j0;
        if (pos >= end) return false;
        j0 = 0;
        if (++hd == heads) {
            hd = 0;
            ++u;
            load(p);
        }
        cut();
        return true;
    }
    __device__ __forceinline__ int tiles() const { return t.n_cnt > 0 ? j1 - j0 : 0; }
    __device__ __forceinline__ bool whole() const { return j0 == 0 && j1 == cc; }
    // of a cut item: the CTA its first position belongs to, and its number of parts
    __device__ __forceinline__ void parts(int& first, int& count) const {
        const long long s = pos - j0;
        first = (int)(s / chunk);
        count = (int)((s + cc - 1) / chunk) - first + 1;
    }
};

// packed_plan.cu
cudaError_t launch_fwd_plan(const PackedFwd& a, const FwdGeom& g, const FwdPlan& p, cudaStream_t st);

// Joins the parts of one cut item (threads tid of nthreads, all of them past the barrier that
// follows the last part's arrival): O = sum_k O_k 2^(m_k - M) / sum_k l_k 2^(m_k - M).
template <typename T>
__device__ __forceinline__ void join_parts(const PackedFwd& a, const FwdPlan& p, const FwdTile& t, int head0, int g,
                                           int rows, int rows_ld, int D, int first, int count, int tid,
                                           int nthreads) {
    const int c4n = a.d / 4;
    for (int e = tid; e < rows * c4n; e += nthreads) {
        const int r = e / c4n, c = (e - r * c4n) * 4;
        float M = -INFINITY;
        for (int k = 0; k < count; ++k) {
            const int slot = k == 0 ? 2 * first + 1 : 2 * (first + k);
            M = fmaxf(M, __ldcg(&p.part_ml[(size_t)slot * rows_ld + r]).x);
        }
        float L = 0.f;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < count; ++k) {
            const int slot = k == 0 ? 2 * first + 1 : 2 * (first + k);
            const float2 ml = __ldcg(&p.part_ml[(size_t)slot * rows_ld + r]);
            const float w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
            if (w == 0.f) continue;  // a part in which the row sees no key
            const float4 o = __ldcg(reinterpret_cast<const float4*>(p.part_o + ((size_t)slot * rows_ld + r) * D + c));
            L += ml.y * w;
            s.x += o.x * w, s.y += o.y * w, s.z += o.z * w, s.w += o.w * w;
        }
        const float inv = L > 0.f ? 1.f / L : 0.f;
        const int tok = t.q_tok + r / g, h = head0 + r % g;
        T out[4] = {TypeTraits<T>::from_f32(s.x * inv), TypeTraits<T>::from_f32(s.y * inv),
                    TypeTraits<T>::from_f32(s.z * inv), TypeTraits<T>::from_f32(s.w * inv)};
        T* dst = static_cast<T*>(a.O) + tok * a.o.tok + h * a.o.head + c;
#pragma unroll
        for (int q = 0; q < 4; ++q) dst[q] = out[q];
        if (c == 0)
            a.LSE[(size_t)h * a.T_q + tok] = L > 0.f ? (M + log2f(L)) * 0.6931471805599453f : -INFINITY;
    }
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

// A 128-row query tile: rows q_tok .. q_tok + rows - 1 of Q; its place in the list is its place
// in the padded rows of the accumulator, D and the LSE copy.
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
    int pad;
};

struct BwdPlan {
    long long* head;      // [0] query tiles, [1] key tiles
    QueryTile* query;     // [max_units]
    KeyTile* key;         // [max_keys], in sequence order
    int* order;           // [max_keys] key tiles, most query tiles first
    int *seq_q, *seq_k;   // [N + 1] first query / key tile of each sequence
    CUtensorMap* maps;    // [N][4] of each sequence: Q, dO, K, V (tensor-core kernel)
    unsigned *sem, *ticket;  // deterministic: turn counters [H][max_units], start-order ticket
    float *lse2, *D;      // [H][rows]
    float* dqacc;         // [rows][H][d] fp32, not scaled
    long long rows;       // max_units * 128
    int max_units, max_keys;
};

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
    q.head = reinterpret_cast<long long*>(take(16));
    q.ticket = reinterpret_cast<unsigned*>(take(4));
    q.sem = reinterpret_cast<unsigned*>(take(a.deterministic ? (size_t)a.H * q.max_units * 4 : 0));
    q.query = reinterpret_cast<QueryTile*>(take((size_t)q.max_units * sizeof(QueryTile)));
    q.key = reinterpret_cast<KeyTile*>(take((size_t)q.max_keys * sizeof(KeyTile)));
    q.order = reinterpret_cast<int*>(take((size_t)q.max_keys * 4));
    q.seq_q = reinterpret_cast<int*>(take(((size_t)a.N + 1) * 4));
    q.seq_k = reinterpret_cast<int*>(take(((size_t)a.N + 1) * 4));
    q.maps = reinterpret_cast<CUtensorMap*>(take(tensor_cores ? (size_t)a.N * 4 * sizeof(CUtensorMap) : 0));
    q.lse2 = reinterpret_cast<float*>(take((size_t)q.rows * a.H * 4));
    q.D = reinterpret_cast<float*>(take((size_t)q.rows * a.H * 4));
    q.dqacc = reinterpret_cast<float*>(take((size_t)q.rows * a.H * a.d * 4));
    if (p) *p = q;
    return at;
}

// packed_plan.cu: tiles, order, maps, counters; with a.fill the gradient rows of no sequence
cudaError_t launch_bwd_plan(const PackedBwd& a, const BwdPlan& p, bool tensor_cores, cudaStream_t st);
// packed_simt.cu: D, the LSE copy and a zeroed accumulator; dQ from the accumulator
cudaError_t launch_packed_preprocess(const PackedBwd& a, const BwdPlan& p, cudaStream_t st);
cudaError_t launch_packed_dq(const PackedBwd& a, const BwdPlan& p, cudaStream_t st);
// packed_bwd.cu (f16 / bf16, head dim <= 128) and packed_bwd_simt.cu (f32, head dim 256)
cudaError_t launch_packed_bwd(const PackedBwd& a, const BwdPlan& p, cudaStream_t st);
cudaError_t launch_packed_bwd_simt(const PackedBwd& a, const BwdPlan& p, cudaStream_t st);

// Map of the fp32 accumulator [rows][H][d]: boxes of 32 columns, one head, 128 rows.
bool bwd_acc_map(CUtensorMap* m, const PackedBwd& a, const BwdPlan& p);

// Orders this thread's later uses of a tensor map after its writes (by an earlier kernel).
__device__ __forceinline__ void tensormap_acquire(const CUtensorMap* m) {
    asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// packed_api.cu: reads the error word of the packed and paged calls on the current device into
// *word and clears it.  Returns an fa_status.
int packed_take_error_word(unsigned int* word);

// ---------------------------------------------------------------- page lookup
// Page that holds key j of a request, or `pages` (one past the cache, which TMA reads as zeros
// and the CUDA-core kernel skips) with *bad set when the table's entry is not a page.
__host__ __device__ __forceinline__ int page_of(const int* row, int j, int page_size, int max_pages, int pages,
                                                bool* bad) {
    const int e = j / page_size;
    const int id = e < max_pages ? row[e] : -1;
    if (id >= 0 && id < pages) return id;
    *bad = true;
    return pages;
}

}  // namespace fa
