// packed_simt.cu -- attention forward over packed sequences or a paged cache on CUDA cores:
// fp32 inputs, and 16-bit ones whose strides, page size or head group the tensor-core kernel's
// TMA boxes cannot address.  The same plan and the same joining of cut items as there; a tile
// is 64 rows (query tokens x heads of one key/value head, packed) by 64 keys, a thread of the
// 16 x 16 grid owns a 4 x 4 block of scores.  fp32 throughout; the online softmax per row.  Bound by the FMA
// pipe's shared-memory operands: 4 x 2048 fp32 tokens, H = 16, d = 64, causal 1.6 ms (21
// TFLOP/s).
#include <math.h>

#include "packed.cuh"

namespace fa {
namespace {

constexpr int BM = 64, BN = 64;
constexpr int kThreads = 256;
constexpr int KT_LD = BN + 4;
constexpr int kOverhead = 1;  // a tile takes longer than the rest of its item

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    packed_fwd_simt_kernel(const PackedFwd a, const FwdPlan plan, int hsub) {
    extern __shared__ float smem[];
    __shared__ int s_last;
    __shared__ float2 s_row[BM];
    float* sQ = smem;             // [BM][D]
    float* sKt = sQ + BM * D;     // [D][KT_LD]
    float* sV = sKt + D * KT_LD;  // [BN][D]
    float* sP = sV + BN * D;      // [BM][BN]
    ptx::griddep_wait();
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    constexpr int CPT = D / 16;
    const int g = a.H / a.H_kv;
    const T* Q = static_cast<const T*>(a.Q);
    const T* K = static_cast<const T*>(a.K);
    const T* V = static_cast<const T*>(a.V);
    FwdShare share;
    share.read(plan, blockIdx.x);
    FwdWalk w;
    for (bool more = w.init(share, blockIdx.x, a.H_kv * hsub, kOverhead); more; more = w.next()) {
        // groups of more heads than a tile has rows are cut into hsub pieces of up to 64
        const int hk = w.hd / hsub, h0 = (w.hd % hsub) * BM;
        const int gh = min(g - h0, BM);      // heads of this item
        const int head0 = hk * g + h0;
        const int rows = w.t.n_tok * gh;
        __syncthreads();
        for (int e = tid; e < BM * D; e += kThreads) {
            const int r = e / D, c = e % D;
            sQ[e] = r < rows ? TypeTraits<T>::to_f32(Q[(long long)(w.t.q_tok + r / gh) * a.q.tok +
                                                       (long long)(head0 + r % gh) * a.q.head + c])
                             : 0.f;
        }
        float m[4], l[4], acc[4][CPT];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
#pragma unroll
            for (int cc = 0; cc < CPT; ++cc) acc[i][cc] = 0.f;
        }
        const int nt = w.tiles();
        const int k_lo = a.window > 0 ? w.t.pos0 - a.window + 1 : 0;  // no row sees an earlier key
        for (int jt = 0; jt < nt; ++jt) {
            const int n0 = (w.t.n_first + w.j0 + jt) * BN;
            __syncthreads();
            for (int e = tid; e < BN * D; e += kThreads) {
                const int r = e / D, c = e % D;
                const int j = n0 + r;
                float kf = 0.f, vf = 0.f;
                if (j < w.t.S_k && j >= k_lo) {
                    long long ko, vo;
                    bool bad = false;
                    if (a.cu_k == nullptr) {
                        const long long pg = page_of(a.table + (size_t)w.t.n * a.max_pages, j, a.page_size,
                                                     a.max_pages, a.pages, &bad);
                        const long long in = j % a.page_size;
                        ko = pg * a.k_page + in * a.k.tok;
                        vo = pg * a.v_page + in * a.v.tok;
                    } else {
                        ko = (long long)(w.t.k_base + j) * a.k.tok;
                        vo = (long long)(w.t.k_base + j) * a.v.tok;
                    }
                    if (bad) {
                        if (c == 0) atomicOr(a.err, kErrPage);
                    } else {
                        kf = TypeTraits<T>::to_f32(K[ko + (long long)hk * a.k.head + c]);
                        vf = TypeTraits<T>::to_f32(V[vo + (long long)hk * a.v.head + c]);
                    }
                }
                sKt[c * KT_LD + r] = kf;
                sV[e] = vf;
            }
            __syncthreads();
            float sc[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int b = 0; b < 4; ++b) sc[i][b] = 0.f;
            for (int c = 0; c < D; ++c) {
                const float4 k4 = *reinterpret_cast<const float4*>(sKt + c * KT_LD + tx * 4);
                const float kv[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float qv = sQ[(ty * 4 + i) * D + c];
#pragma unroll
                    for (int b = 0; b < 4; ++b) sc[i][b] = fmaf(qv, kv[b], sc[i][b]);
                }
            }
            // scores in log2 units
            const float sl2 = a.scale * 1.4426950408889634f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = ty * 4 + i;
                const int p = w.t.pos0 + r / gh;
                float rmax = -INFINITY;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const int j = n0 + tx * 4 + b;
                    const bool vis = j < w.t.S_k && key_visible(p, j, a.causal, a.window);
                    sc[i][b] = vis ? sc[i][b] * sl2 : -INFINITY;
                    rmax = fmaxf(rmax, sc[i][b]);
                }
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) rmax = fmaxf(rmax, __shfl_xor_sync(0xffffffffu, rmax, o, 16));
                const float mn = fmaxf(m[i], rmax);
                // no max yet: a masked score gives exp2(-inf) = 0, a NaN one (left out of the max) NaN
                const float base = mn == -INFINITY ? 0.f : mn;
                const float alpha = mn == -INFINITY ? 1.f : exp2f(m[i] - mn);
                float rs = 0.f;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const float pv = exp2f(sc[i][b] - base);
                    sP[r * BN + tx * 4 + b] = pv;
                    rs += pv;
                }
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) rs += __shfl_xor_sync(0xffffffffu, rs, o, 16);
                l[i] = l[i] * alpha + rs;
                m[i] = mn;
#pragma unroll
                for (int cc = 0; cc < CPT; ++cc) acc[i][cc] *= alpha;
            }
            __syncthreads();
            for (int j = 0; j < BN; ++j) {
                float vv[CPT];
#pragma unroll
                for (int cc = 0; cc < CPT; ++cc) vv[cc] = sV[j * D + tx + 16 * cc];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float pv = sP[(ty * 4 + i) * BN + j];
#pragma unroll
                    for (int cc = 0; cc < CPT; ++cc) acc[i][cc] = fmaf(pv, vv[cc], acc[i][cc]);
                }
            }
        }
        const bool whole = w.whole();
        const int slot = 2 * (int)blockIdx.x + (w.j0 == 0 ? 1 : 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = ty * 4 + i;
            if (r >= rows) continue;
            const int tok = w.t.q_tok + r / gh, head = head0 + r % gh;
            if (whole) {
                const float inv = inv_sum(l[i]);
                T* Orow = static_cast<T*>(a.O) + (long long)tok * a.o.tok + (long long)head * a.o.head;
#pragma unroll
                for (int cc = 0; cc < CPT; ++cc)  // without a key acc is 0 times V, NaN where V is infinite
                    Orow[tx + 16 * cc] = TypeTraits<T>::from_f32(l[i] == 0.f ? 0.f : acc[i][cc] * inv);
                if (tx == 0) a.LSE[(size_t)head * a.T_q + tok] = lse_of(m[i], l[i]);
            } else {
                float* Prow = plan.part_o + ((size_t)slot * BM + r) * D;
#pragma unroll
                for (int cc = 0; cc < CPT; ++cc) Prow[tx + 16 * cc] = acc[i][cc];
                if (tx == 0) plan.part_ml[(size_t)slot * BM + r] = make_float2(part_max(m[i], l[i]), l[i]);
            }
        }
        if (!whole) {  // the last part to arrive joins the item
            int first, count;
            w.parts(first, count);
            __threadfence();
            __syncthreads();
            if (tid == 0) s_last = arrive_part(&plan.done[first], plan.tag, count);
            __syncthreads();
            if (s_last) {
                __threadfence();
                join_parts<T, kThreads, BM, D, 8>(a, plan, w.t, head0, gh, rows, first, count, tid, s_row,
                                               [] { __syncthreads(); });
            }
        }
    }
}

template <typename T, int D>
cudaError_t launch_t(const PackedFwd& a, void* ws, size_t* bytes, cudaStream_t st) {
    const size_t smem = sizeof(float) * (BM * D + D * KT_LD + BN * D + BM * BN);
    auto kern = packed_fwd_simt_kernel<T, D>;
    const int g = a.H / a.H_kv;
    const int hsub = (g + BM - 1) / BM;
    FwdGeom geo;
    geo.rows = BM;
    geo.tpt = g < BM ? BM / g : 1;
    geo.bn = BN;
    geo.heads = a.H_kv * hsub;
    geo.ctas = sm_count() * (D <= 96 ? 2 : 1);  // resident CTAs by shared memory
    geo.D = D;
    geo.min_chunk = 2;
    geo.overhead = kOverhead;
    geo.self = false;
    FwdPlan plan;
    *bytes = fwd_plan_layout(a, geo, ws, &plan);
    if (ws == nullptr) return cudaSuccess;
    plan.tag = next_tag();
    cudaError_t e = launch_fwd_plan(a, geo, plan, st);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kern<<<geo.ctas, kThreads, smem, st>>>(a, plan, hsub);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_packed_fwd_simt(const PackedFwd& a, void* ws, size_t* bytes, cudaStream_t st) {
#define FA_L(T, DD) return launch_t<T, DD>(a, ws, bytes, st)
    FA_DISPATCH_HEAD_DIM(a.dtype, a.d, FA_L);
#undef FA_L
    return cudaErrorInvalidValue;
}

}  // namespace fa
