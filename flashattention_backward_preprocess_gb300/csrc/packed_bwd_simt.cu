// packed_bwd_simt.cu -- the passes around the packed backward's main kernel, and that kernel
// on CUDA cores (fp32 inputs).
//
// Preprocess, per query row and head: D = sum_c dO_c O_c (fp32), LSE * log2 e into rows padded
// to whole query tiles (+inf on padding rows and rows without keys, so their P is 0; the NaN of a
// row that sees one stays, and makes its P NaN), and the row of the fp32 dQ accumulator set to
// zero.  dQ: scale times the accumulator, rounded once.  Both read and write each byte once.  For
// 11390 bf16 tokens of H = 32, d = 128 the first moves 374 MB in 61 us, 320 of them at DRAM (5.2
// TB/s; the rest of the zeroed accumulator is still in L2), the second 280 MB in 40 us, 239 of
// them at DRAM (6.0 TB/s, 0.88 of the measured copy rate; the rest of dQ is still in L2).
//
// Main kernel (the mathematics of bwd_simt.cu): one CTA owns BN key rows of one (sequence, kv
// head), dK and dV in registers, and walks BM-row query tiles of every query head of the group;
// every product is a register-tiled block product from shared memory in fp32.  Bound by the
// FMA pipe and its shared-memory operands: 4 x 4 scores of a thread need 24 shared-memory
// wavefronts a warp for 32 issue cycles of FMA.  5 sequences of 1 to 1024 fp32 tokens (2122 in
// all), H = 8, H_kv = 2, d = 128, causal: 352 us a call, 466 us with 512 threads of 2 x 4
// scores; 4 x 2048 tokens, H = 16, d = 64 3.2 ms (27 TFLOP/s), deterministic 4.2 ms.
#include <math.h>

#include "packed.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;

constexpr int lanes_per_row(int chunks) {
    int l = 1;
    while (l < chunks && l < 32) l *= 2;
    return l;
}

constexpr int kRowsPerBlock = 8;  // tile rows of one block; its rows are kRowsPerBlock x H
constexpr int kBatch = 4;         // rows whose loads a thread has in flight together

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) packed_preprocess_kernel(const PackedBwd a, const BwdPlan p) {
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    constexpr int VEC = 16 / sizeof(T);
    constexpr int CPR = D / VEC;
    constexpr int LPR = lanes_per_row(CPR);
    const int u = blockIdx.x / (kBwdTile / kRowsPerBlock);
    if (u >= p.head[0]) return;
    const int r0 = (blockIdx.x % (kBwdTile / kRowsPerBlock)) * kRowsPerBlock;
    const QueryTile t = p.query[u];
    const int lane = threadIdx.x % LPR;
    const int total = kRowsPerBlock * a.H;
    // groups of LPR lanes take a row each; kBatch rows' loads go out before the first is used
    constexpr int G = kThreads / LPR, CH = (CPR + LPR - 1) / LPR;  // rows per step, pieces per lane
    for (int e0 = 0; e0 < total; e0 += kBatch * G) {
        int4 x[kBatch][CH], y[kBatch][CH];
        float acc[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int e = e0 + b * G + threadIdx.x / LPR, r = r0 + e / a.H, h = e % a.H;
            const bool valid = e < total && r < t.rows;
            const T* dO = static_cast<const T*>(a.dO) + (long long)(t.q_tok + r) * a.sdo.tok + (long long)h * a.sdo.head;
            const T* O = static_cast<const T*>(a.O) + (long long)(t.q_tok + r) * a.so.tok + (long long)h * a.so.head;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int ch = lane + c * LPR;
                const bool in = valid && (CPR % LPR == 0 || ch < CPR);
                x[b][c] = in ? __ldcs(reinterpret_cast<const int4*>(dO) + ch) : make_int4(0, 0, 0, 0);
                y[b][c] = in ? __ldcs(reinterpret_cast<const int4*>(O) + ch) : make_int4(0, 0, 0, 0);
            }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int e = e0 + b * G + threadIdx.x / LPR, r = r0 + e / a.H, h = e % a.H;
            const bool valid = e < total && r < t.rows;
            float* z = p.dqacc + (((long long)t.q_tok + r) * a.H + h) * D;
            acc[b] = 0.f;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int ch = lane + c * LPR;
                const T* tx = reinterpret_cast<const T*>(&x[b][c]);
                const T* ty = reinterpret_cast<const T*>(&y[b][c]);
#pragma unroll
                for (int k = 0; k < VEC; ++k)
                    acc[b] = fmaf(TypeTraits<T>::to_f32(tx[k]), TypeTraits<T>::to_f32(ty[k]), acc[b]);
                if (valid && (CPR % LPR == 0 || ch < CPR)) {
#pragma unroll
                    for (int k = 0; k < VEC / 4; ++k)
                        reinterpret_cast<float4*>(z)[ch * (VEC / 4) + k] = make_float4(0.f, 0.f, 0.f, 0.f);
                }
            }
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) acc[b] += __shfl_xor_sync(0xffffffffu, acc[b], o, LPR);
            if (e < total && lane == 0) {
                const long long row = h * p.rows + (long long)u * kBwdTile + r;
                const float l = valid ? a.LSE[(size_t)h * a.T_q + t.q_tok + r] : -INFINITY;
                p.D[row] = acc[b];
                p.lse2[row] = l == -INFINITY ? INFINITY : l * 1.4426950408889634f;
            }
        }
    }
}

template <typename T>
__device__ __forceinline__ float4 load4(const T* p) {
    if constexpr (sizeof(T) == 4) {
        return *reinterpret_cast<const float4*>(p);
    } else {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        const T* t = reinterpret_cast<const T*>(&u);
        return make_float4(TypeTraits<T>::to_f32(t[0]), TypeTraits<T>::to_f32(t[1]), TypeTraits<T>::to_f32(t[2]),
                           TypeTraits<T>::to_f32(t[3]));
    }
}
template <typename T>
__device__ __forceinline__ void store4(T* p, float x, float y, float z, float w) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(x, y, z, w);
    } else {
        alignas(8) T t[4] = {TypeTraits<T>::from_f32(x), TypeTraits<T>::from_f32(y), TypeTraits<T>::from_f32(z),
                             TypeTraits<T>::from_f32(w)};
        *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(t);
    }
}

constexpr int kCutBlocks = 8;  // blocks per cut key tile and head

// dK and dV of a cut key tile: its parts' sums, added in order.
template <typename T, int D>
__device__ void join_cut(const PackedBwd& a, const BwdPlan& p, int b) {
    constexpr int C4 = D / 4, kRows = kBwdTile / kCutBlocks;
    const int i = b / kCutBlocks / a.H_kv, hk = b / kCutBlocks % a.H_kv;
    if (i >= p.head[2]) return;
    const KeyWork w = p.cut[i];
    const KeyTile kt = p.key[w.tile];
    const int r0 = b % kCutBlocks * kRows, rows = min(kRows, min(kBwdTile, kt.S_k - kt.n0) - r0);
    const size_t step = (size_t)a.H_kv * 2 * kBwdTile * D;  // from a part to the next
    for (int e = threadIdx.x; e < rows * 2 * C4; e += kThreads) {
        const int c = e % C4, which = e / C4 % 2, r = r0 + e / (2 * C4);
        const float4* s = reinterpret_cast<const float4*>(
                              p.part + (((size_t)w.slot * a.H_kv + hk) * 2 + which) * kBwdTile * D + (size_t)r * D) + c;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = 0; k < w.parts; ++k) {
            const float4 y = __ldcs(s + k * (step / 4));
            x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
        }
        const float f = which ? a.scale : 1.f;
        const RowStride str = which ? a.sdk : a.sdv;
        T* dst = static_cast<T*>(which ? a.dK : a.dV) + (long long)(kt.k_tok + r) * str.tok + (long long)hk * str.head;
        store4<T>(dst + 4 * c, x.x * f, x.y * f, x.z * f, x.w * f);
    }
}

// Blocks [0, dq_blocks): dQ rows; the rest: cut key tiles.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) packed_dq_kernel(const PackedBwd a, const BwdPlan p, int dq_blocks) {
    ptx::griddep_wait();
    if ((int)blockIdx.x >= dq_blocks) {
        join_cut<T, D>(a, p, blockIdx.x - dq_blocks);
        return;
    }
    constexpr int C8 = D / 8;  // 8-column groups per row
    const int u = blockIdx.x / (kBwdTile / kRowsPerBlock);
    if (u >= p.head[0]) return;
    const int r0 = (blockIdx.x % (kBwdTile / kRowsPerBlock)) * kRowsPerBlock;
    const QueryTile t = p.query[u];
    const int rows = min(kRowsPerBlock, t.rows - r0);
    const int total = rows * a.H * C8;
    for (int e0 = threadIdx.x; e0 < total; e0 += kBatch * kThreads) {
        float4 x[kBatch], y[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int e = e0 + b * kThreads;
            if (e < total) {
                // rows of the block are consecutive in the accumulator
                const float4* s = reinterpret_cast<const float4*>(p.dqacc + ((long long)t.q_tok + r0) * a.H * D) + 2ll * e;
                x[b] = __ldcs(s);
                y[b] = __ldcs(s + 1);
            }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int e = e0 + b * kThreads;
            if (e >= total) break;
            const int c = e % C8, rh = e / C8;
            const int r = r0 + rh / a.H, h = rh % a.H;
            const float v[8] = {x[b].x, x[b].y, x[b].z, x[b].w, y[b].x, y[b].y, y[b].z, y[b].w};
            T* dst = static_cast<T*>(a.dQ) + (long long)(t.q_tok + r) * a.sdq.tok + (long long)h * a.sdq.head + 8 * c;
            if constexpr (sizeof(T) == 4) {
                float4* o = reinterpret_cast<float4*>(dst);
                o[0] = make_float4(v[0] * a.scale, v[1] * a.scale, v[2] * a.scale, v[3] * a.scale);
                o[1] = make_float4(v[4] * a.scale, v[5] * a.scale, v[6] * a.scale, v[7] * a.scale);
            } else {
                alignas(16) T o[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) o[k] = TypeTraits<T>::from_f32(v[k] * a.scale);
                __stcs(reinterpret_cast<int4*>(dst), *reinterpret_cast<const int4*>(o));
            }
        }
    }
}

template <int D>
struct SCfg {
    static constexpr int BN = D <= 128 ? 64 : 32;  // key rows per CTA (shared memory at d = 256)
    static constexpr int BM = BN;
    static constexpr int LD = D + 4;
    static constexpr int LP = BN + 4;
    static constexpr int TR = BM / 16;
    static constexpr int TC = BN / 16;
    static constexpr int NG = (D / 4 + 15) / 16;
    static constexpr size_t SMEM = sizeof(float) * ((size_t)(2 * BN + 2 * BM) * LD + 2 * BM * LP + 2 * BM);
};

// rows [0, n) of a tile (row stride `ld` elements) into a padded fp32 shared tile; zeros behind
template <typename T, int D>
__device__ __forceinline__ void stage_rows(float* dst, const T* src, long long ld, int n, int rows) {
    constexpr int LD = D + 4;
    for (int e = threadIdx.x; e < rows * (D / 4); e += kThreads) {
        const int r = e / (D / 4), c4 = e % (D / 4);
        const float4 v = r < n ? load4(src + r * ld + 4 * c4) : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4*>(dst + r * LD + 4 * c4) = v;
    }
}

// S and dP blocks: rows ty + 16r of Q and dO, keys tx + 16c, 4 head-dim columns a step.
template <int D, int TR, int TC>
__device__ __forceinline__ void block_products(const float* sQ, const float* sdO, const float* sK, const float* sV, int ty,
                                               int tx, float (&accS)[TR][TC], float (&accP)[TR][TC]) {
    constexpr int LD = SCfg<D>::LD;
#pragma unroll
    for (int r = 0; r < TR; ++r)
#pragma unroll
        for (int c = 0; c < TC; ++c) accS[r][c] = accP[r][c] = 0.f;
#pragma unroll 4
    for (int k = 0; k < D; k += 4) {
        float4 q[TR], o[TR], kk[TC], v[TC];
#pragma unroll
        for (int r = 0; r < TR; ++r) {
            q[r] = *reinterpret_cast<const float4*>(sQ + (ty + 16 * r) * LD + k);
            o[r] = *reinterpret_cast<const float4*>(sdO + (ty + 16 * r) * LD + k);
        }
#pragma unroll
        for (int c = 0; c < TC; ++c) {
            kk[c] = *reinterpret_cast<const float4*>(sK + (tx + 16 * c) * LD + k);
            v[c] = *reinterpret_cast<const float4*>(sV + (tx + 16 * c) * LD + k);
        }
#pragma unroll
        for (int r = 0; r < TR; ++r)
#pragma unroll
            for (int c = 0; c < TC; ++c) {
                accS[r][c] = fmaf(q[r].x, kk[c].x, accS[r][c]);
                accS[r][c] = fmaf(q[r].y, kk[c].y, accS[r][c]);
                accS[r][c] = fmaf(q[r].z, kk[c].z, accS[r][c]);
                accS[r][c] = fmaf(q[r].w, kk[c].w, accS[r][c]);
                accP[r][c] = fmaf(o[r].x, v[c].x, accP[r][c]);
                accP[r][c] = fmaf(o[r].y, v[c].y, accP[r][c]);
                accP[r][c] = fmaf(o[r].z, v[c].z, accP[r][c]);
                accP[r][c] = fmaf(o[r].w, v[c].w, accP[r][c]);
            }
    }
}

// accQ += dS K: query rows ty + 16r, column groups tx + 16q, keys in order.
template <int D, int TR, int NG, int BN>
__device__ __forceinline__ void add_ds_k(const float* sdS, const float* sK, int ty, int tx, float (&accQ)[TR][NG][4]) {
    constexpr int LD = SCfg<D>::LD, LP = SCfg<D>::LP;
#pragma unroll 2
    for (int jj = 0; jj < BN; ++jj) {
        float ds[TR];
#pragma unroll
        for (int r = 0; r < TR; ++r) ds[r] = sdS[(ty + 16 * r) * LP + jj];
#pragma unroll
        for (int q = 0; q < NG; ++q) {
            const int f = tx + 16 * q;
            if (NG * 16 * 4 == D || f < D / 4) {
                const float4 kv = *reinterpret_cast<const float4*>(sK + jj * LD + 4 * f);
#pragma unroll
                for (int r = 0; r < TR; ++r) {
                    accQ[r][q][0] = fmaf(ds[r], kv.x, accQ[r][q][0]);
                    accQ[r][q][1] = fmaf(ds[r], kv.y, accQ[r][q][1]);
                    accQ[r][q][2] = fmaf(ds[r], kv.z, accQ[r][q][2]);
                    accQ[r][q][3] = fmaf(ds[r], kv.w, accQ[r][q][3]);
                }
            }
        }
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) packed_bwd_simt_kernel(const PackedBwd a, const BwdPlan p) {
    using C = SCfg<D>;
    constexpr int BN = C::BN, BM = C::BM, LD = C::LD, LP = C::LP, TR = C::TR, TC = C::TC, NG = C::NG;
    constexpr int kPieces = kBwdTile / BN;  // CTAs per work and head (bwd_pieces)
    extern __shared__ float4 smem4[];
    float* smem = reinterpret_cast<float*>(smem4);
    float* sK = smem;
    float* sV = sK + BN * LD;
    float* sQ = sV + BN * LD;
    float* sdO = sQ + BM * LD;
    float* sP = sdO + BM * LD;
    float* sdS = sP + BM * LP;
    float* sL = sdS + BM * LP;
    float* sDd = sL + BM;
    ptx::griddep_wait();

    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int item = blockIdx.x / kPieces;
    if (item / a.H_kv >= p.head[1]) return;
    const KeyWork work = p.work[item / a.H_kv];
    const KeyTile kt = p.key[work.tile];
    const int hk = item % a.H_kv, g = a.H / a.H_kv;
    const int sub = (blockIdx.x % kPieces) * BN;  // this CTA's rows within the plan tile
    const int n0 = kt.n0 + sub, S_q = kt.S_q, S_k = kt.S_k;
    if (n0 >= S_k) return;
    const int off = S_k - S_q;
    const float sc2 = a.scale * 1.4426950408889634f;
    const int krows = min(BN, S_k - n0);
    stage_rows<T, D>(sK, static_cast<const T*>(a.K) + (long long)(kt.k_tok + sub) * a.sk.tok + (long long)hk * a.sk.head,
                     a.sk.tok, krows, BN);
    stage_rows<T, D>(sV, static_cast<const T*>(a.V) + (long long)(kt.k_tok + sub) * a.sv.tok + (long long)hk * a.sv.head,
                     a.sv.tok, krows, BN);

    float accV[TC][NG][4], accK[TC][NG][4];
#pragma unroll
    for (int r = 0; r < TC; ++r)
#pragma unroll
        for (int q = 0; q < NG; ++q)
#pragma unroll
            for (int u = 0; u < 4; ++u) accV[r][q][u] = accK[r][q][u] = 0.f;

    Shape sh;
    sh.S_q = S_q;
    sh.S_k = S_k;
    sh.causal = a.causal;
    sh.window = a.window;
    int i_begin, i_end;
    query_range(sh, n0, min(n0 + BN, S_k), i_begin, i_end);
    const int m_first = i_begin / BM * BM;
    const int nq = i_end > i_begin ? (i_end - m_first + BM - 1) / BM : 0;
    const long long q_tok0 = kt.q_tok;                      // first query row of the sequence
    const long long row0 = (long long)kt.unit0 * kBwdTile;  // and in the padded rows
    // this CTA's share of the iterations (all of them unless the tile is cut)
    const int it_lo = (int)((long long)g * nq * work.part / work.parts);
    const int it_hi = (int)((long long)g * nq * (work.part + 1) / work.parts);
    for (int it = it_lo; it < it_hi; ++it) {
        const int h = hk * g + it / nq;
        const int m0 = m_first + (it % nq) * BM;
        const int rows = min(BM, S_q - m0);
        __syncthreads();  // the previous step's reads are done
        stage_rows<T, D>(sQ, static_cast<const T*>(a.Q) + (q_tok0 + m0) * a.sq.tok + (long long)h * a.sq.head, a.sq.tok,
                         rows, BM);
        stage_rows<T, D>(sdO, static_cast<const T*>(a.dO) + (q_tok0 + m0) * a.sdo.tok + (long long)h * a.sdo.head,
                         a.sdo.tok, rows, BM);
        for (int r = tid; r < BM; r += kThreads) {
            sL[r] = p.lse2[h * p.rows + row0 + m0 + r];  // +inf on padding rows: P = 0
            sDd[r] = p.D[h * p.rows + row0 + m0 + r];
        }
        __syncthreads();
        // ---- S and dP blocks (rows ty + 16r, keys tx + 16c), 4 head-dim columns a step
        float accS[TR][TC], accP[TR][TC];
        block_products<D, TR, TC>(sQ, sdO, sK, sV, ty, tx, accS, accP);
        // ---- P = exp(scale S - LSE) on visible pairs, dS = P (dP - D)
#pragma unroll
        for (int r = 0; r < TR; ++r) {
            const int ri = ty + 16 * r, i = m0 + ri;
            const float l2 = sL[ri], Di = sDd[ri];
#pragma unroll
            for (int c = 0; c < TC; ++c) {
                const int j = n0 + tx + 16 * c;
                const bool vis = i < S_q && j < S_k && key_visible(i + off, j, a.causal, a.window);
                const float pv = vis ? exp2f(fmaf(accS[r][c], sc2, -l2)) : 0.f;
                sP[ri * LP + tx + 16 * c] = pv;
                sdS[ri * LP + tx + 16 * c] = pv * (accP[r][c] - Di);
            }
        }
        __syncthreads();
        // ---- dV += P^T dO, dK += dS^T Q (key rows ty + 16r, column groups tx + 16q)
#pragma unroll 2
        for (int i = 0; i < BM; ++i) {
            float pk[TC], dk[TC];
#pragma unroll
            for (int r = 0; r < TC; ++r) {
                pk[r] = sP[i * LP + ty + 16 * r];
                dk[r] = sdS[i * LP + ty + 16 * r];
            }
#pragma unroll
            for (int q = 0; q < NG; ++q) {
                const int f = tx + 16 * q;
                if (NG * 16 * 4 == D || f < D / 4) {
                    const float4 o = *reinterpret_cast<const float4*>(sdO + i * LD + 4 * f);
                    const float4 x = *reinterpret_cast<const float4*>(sQ + i * LD + 4 * f);
#pragma unroll
                    for (int r = 0; r < TC; ++r) {
                        accV[r][q][0] = fmaf(pk[r], o.x, accV[r][q][0]);
                        accV[r][q][1] = fmaf(pk[r], o.y, accV[r][q][1]);
                        accV[r][q][2] = fmaf(pk[r], o.z, accV[r][q][2]);
                        accV[r][q][3] = fmaf(pk[r], o.w, accV[r][q][3]);
                        accK[r][q][0] = fmaf(dk[r], x.x, accK[r][q][0]);
                        accK[r][q][1] = fmaf(dk[r], x.y, accK[r][q][1]);
                        accK[r][q][2] = fmaf(dk[r], x.z, accK[r][q][2]);
                        accK[r][q][3] = fmaf(dk[r], x.w, accK[r][q][3]);
                    }
                }
            }
        }
        // ---- dQacc += dS K (query rows ty + 16r, column groups tx + 16q)
        if (!a.deterministic) {
            float accQ[TR][NG][4];
#pragma unroll
            for (int r = 0; r < TR; ++r)
#pragma unroll
                for (int q = 0; q < NG; ++q)
#pragma unroll
                    for (int u = 0; u < 4; ++u) accQ[r][q][u] = 0.f;
            add_ds_k<D, TR, NG, BN>(sdS, sK, ty, tx, accQ);
#pragma unroll
            for (int r = 0; r < TR; ++r) {
                const int ri = ty + 16 * r;
                if (ri < rows) {
#pragma unroll
                    for (int q = 0; q < NG; ++q) {
                        const int f = tx + 16 * q;
                        if (NG * 16 * 4 == D || f < D / 4)
                            ptx::red_add_v4(p.dqacc + ((q_tok0 + m0 + ri) * a.H + h) * D + 4 * f, accQ[r][q][0],
                                            accQ[r][q][1], accQ[r][q][2], accQ[r][q][3]);
                    }
                }
            }
        }
    }
    // ---- dK (scaled) and dV rows of this tile
#pragma unroll
    for (int r = 0; r < TC; ++r) {
        const int rr = ty + 16 * r;
        if (rr >= krows) continue;
        T* dV = static_cast<T*>(a.dV) + (long long)(kt.k_tok + sub + rr) * a.sdv.tok + (long long)hk * a.sdv.head;
        T* dK = static_cast<T*>(a.dK) + (long long)(kt.k_tok + sub + rr) * a.sdk.tok + (long long)hk * a.sdk.head;
        float* part = p.part + (((size_t)work.slot * a.H_kv + hk) * 2 * kBwdTile + sub + rr) * D;
#pragma unroll
        for (int q = 0; q < NG; ++q) {
            const int f = tx + 16 * q;
            if (!(NG * 16 * 4 == D || f < D / 4)) continue;
            if (work.parts > 1) {  // one part's sums, added up by the last pass
                store4<float>(part + 4 * f, accV[r][q][0], accV[r][q][1], accV[r][q][2], accV[r][q][3]);
                store4<float>(part + kBwdTile * D + 4 * f, accK[r][q][0], accK[r][q][1], accK[r][q][2], accK[r][q][3]);
                continue;
            }
            store4<T>(dV + 4 * f, accV[r][q][0], accV[r][q][1], accV[r][q][2], accV[r][q][3]);
            store4<T>(dK + 4 * f, accK[r][q][0] * a.scale, accK[r][q][1] * a.scale, accK[r][q][2] * a.scale,
                      accK[r][q][3] * a.scale);
        }
    }
}

// Deterministic dQ of fp32 inputs and of head dim 256: one CTA per (BM query rows, head) forms the
// accumulator rows itself, visiting the key tiles in index order, so every row is one fixed
// sequence of additions.  The block products are those of the main kernel.
template <int D>
constexpr size_t dq_smem() {
    using C = SCfg<D>;
    return sizeof(float) * ((size_t)(2 * C::BN + 2 * C::BM) * C::LD + C::BM * C::LP);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) packed_dq_simt_kernel(const PackedBwd a, const BwdPlan p) {
    using C = SCfg<D>;
    constexpr int BN = C::BN, BM = C::BM, LD = C::LD, LP = C::LP, TR = C::TR, TC = C::TC, NG = C::NG;
    extern __shared__ float4 smem4[];
    float* sK = reinterpret_cast<float*>(smem4);
    float* sV = sK + BN * LD;
    float* sQ = sV + BN * LD;
    float* sdO = sQ + BM * LD;
    float* sdS = sdO + BM * LD;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int u = blockIdx.x / (kBwdTile / BM);
    if (u >= p.head[0]) return;
    const QueryTile t = p.query[u];
    const int r0 = (blockIdx.x % (kBwdTile / BM)) * BM;  // within the query tile
    const int rows = min(BM, t.rows - r0);
    if (rows <= 0) return;
    // the sequence of this query tile
    int n = 0;
    for (int hi = a.N; hi - n > 1;) {
        const int mid = (n + hi) >> 1;
        if (p.seq_q[mid] <= u)
            n = mid;
        else
            hi = mid;
    }
    const int k_tok0 = a.cu_k[n], S_k = a.cu_k[n + 1] - k_tok0;
    const int S_q = a.cu_q[n + 1] - a.cu_q[n];
    const int m0 = t.q_tok - a.cu_q[n] + r0;  // first query of this CTA within the sequence
    const int h = blockIdx.y, hk = h / (a.H / a.H_kv);
    const int off = S_k - S_q;
    const float sc2 = a.scale * 1.4426950408889634f;
    const long long row = (long long)u * kBwdTile + r0;  // in the padded rows
    float* const acc = p.dqacc + (((long long)t.q_tok + r0) * a.H + h) * D;
    stage_rows<T, D>(sQ, static_cast<const T*>(a.Q) + (long long)(t.q_tok + r0) * a.sq.tok + (long long)h * a.sq.head,
                     a.sq.tok, rows, BM);
    stage_rows<T, D>(sdO, static_cast<const T*>(a.dO) + (long long)(t.q_tok + r0) * a.sdo.tok + (long long)h * a.sdo.head,
                     a.sdo.tok, rows, BM);
    float l2[TR], Di[TR], accQ[TR][NG][4];
#pragma unroll
    for (int r = 0; r < TR; ++r) {
        l2[r] = p.lse2[h * p.rows + row + ty + 16 * r];
        Di[r] = p.D[h * p.rows + row + ty + 16 * r];
#pragma unroll
        for (int q = 0; q < NG; ++q)
#pragma unroll
            for (int e = 0; e < 4; ++e) accQ[r][q][e] = 0.f;
    }
    Shape sh;
    sh.S_q = S_q;
    sh.S_k = S_k;
    sh.causal = a.causal;
    sh.window = a.window;
    int k_lo, k_hi;
    key_range(sh, m0, m0 + rows, k_lo, k_hi);
    for (int n0 = k_lo / BN * BN; n0 < k_hi; n0 += BN) {
        __syncthreads();  // the previous step's reads are done
        const int krows = min(BN, S_k - n0);
        stage_rows<T, D>(sK, static_cast<const T*>(a.K) + (long long)(k_tok0 + n0) * a.sk.tok + (long long)hk * a.sk.head,
                         a.sk.tok, krows, BN);
        stage_rows<T, D>(sV, static_cast<const T*>(a.V) + (long long)(k_tok0 + n0) * a.sv.tok + (long long)hk * a.sv.head,
                         a.sv.tok, krows, BN);
        __syncthreads();
        float accS[TR][TC], accP[TR][TC];
        block_products<D, TR, TC>(sQ, sdO, sK, sV, ty, tx, accS, accP);
#pragma unroll
        for (int r = 0; r < TR; ++r) {
            const int ri = ty + 16 * r;
#pragma unroll
            for (int c = 0; c < TC; ++c) {
                const int j = n0 + tx + 16 * c;
                const bool vis = ri < rows && j < S_k && key_visible(m0 + ri + off, j, a.causal, a.window);
                sdS[ri * LP + tx + 16 * c] = vis ? exp2f(fmaf(accS[r][c], sc2, -l2[r])) * (accP[r][c] - Di[r]) : 0.f;
            }
        }
        __syncthreads();
        add_ds_k<D, TR, NG, BN>(sdS, sK, ty, tx, accQ);
    }
#pragma unroll
    for (int r = 0; r < TR; ++r) {
        const int ri = ty + 16 * r;
        if (ri >= rows) continue;
#pragma unroll
        for (int q = 0; q < NG; ++q) {
            const int f = tx + 16 * q;
            if (NG * 16 * 4 == D || f < D / 4)
                *reinterpret_cast<float4*>(acc + (long long)ri * a.H * D + 4 * f) =
                    make_float4(accQ[r][q][0], accQ[r][q][1], accQ[r][q][2], accQ[r][q][3]);
        }
    }
}

template <typename... A>
cudaError_t launch_pdl(void (*k)(A...), long long grid, int threads, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, args...);
}

template <typename T, int D>
cudaError_t preprocess_t(const PackedBwd& a, const BwdPlan& p, cudaStream_t st) {
    return launch_pdl(packed_preprocess_kernel<T, D>, (long long)p.max_units * (kBwdTile / kRowsPerBlock), kThreads, st, a, p);
}

template <typename T, int D>
cudaError_t dq_t(const PackedBwd& a, const BwdPlan& p, cudaStream_t st) {
    const int dq = p.max_units * (kBwdTile / kRowsPerBlock);
    return launch_pdl(packed_dq_kernel<T, D>, dq + (long long)p.max_cut * a.H_kv * kCutBlocks, kThreads, st, a, p, dq);
}

template <typename T, int D>
cudaError_t bwd_t(const PackedBwd& a, const BwdPlan& p, cudaStream_t st) {
    using C = SCfg<D>;
    static std::atomic<uint64_t> ready{0};
    cudaError_t e;
    if (p.max_keys > 0) {
        auto kern = packed_bwd_simt_kernel<T, D>;
        if ((e = allow_smem(kern, (int)C::SMEM, ready)) != cudaSuccess) return e;
        kern<<<(unsigned)((long long)p.max_work * a.H_kv * (kBwdTile / C::BN)), kThreads, C::SMEM, st>>>(a, p);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <typename T, int D>
cudaError_t dq_ordered_t(const PackedBwd& a, const BwdPlan& p, cudaStream_t st) {
    auto kern = packed_dq_simt_kernel<T, D>;
    static std::atomic<uint64_t> ready{0};
    cudaError_t e = allow_smem(kern, (int)dq_smem<D>(), ready);
    if (e != cudaSuccess) return e;
    kern<<<dim3((unsigned)(p.max_units * (kBwdTile / SCfg<D>::BM)), (unsigned)a.H), kThreads, dq_smem<D>(), st>>>(a, p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_packed_preprocess(const PackedBwd& a, const BwdPlan& p, cudaStream_t st) {
    if (p.max_units == 0) return cudaSuccess;
#define FA_L(T, DD) return preprocess_t<T, DD>(a, p, st)
    FA_DISPATCH_HEAD_DIM(a.dtype, a.d, FA_L);
#undef FA_L
    return cudaErrorInvalidValue;
}

cudaError_t launch_packed_dq(const PackedBwd& a, const BwdPlan& p, cudaStream_t st) {
#define FA_L(T, DD) return dq_t<T, DD>(a, p, st)
    FA_DISPATCH_HEAD_DIM(a.dtype, a.d, FA_L);
#undef FA_L
    return cudaErrorInvalidValue;
}

cudaError_t launch_packed_bwd_simt(const PackedBwd& a, const BwdPlan& p, cudaStream_t st) {
    switch (a.d) {
        case 32: return bwd_t<float, 32>(a, p, st);
        case 64: return bwd_t<float, 64>(a, p, st);
        case 96: return bwd_t<float, 96>(a, p, st);
        case 128: return bwd_t<float, 128>(a, p, st);
        case 256: return bwd_t<float, 256>(a, p, st);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_packed_dq_ordered(const PackedBwd& a, const BwdPlan& p, cudaStream_t st) {
    if (p.max_units == 0) return cudaSuccess;
    if (a.dtype == FA_F16) return dq_ordered_t<__half, 256>(a, p, st);
    if (a.dtype == FA_BF16) return dq_ordered_t<__nv_bfloat16, 256>(a, p, st);
    switch (a.d) {
        case 32: return dq_ordered_t<float, 32>(a, p, st);
        case 64: return dq_ordered_t<float, 64>(a, p, st);
        case 96: return dq_ordered_t<float, 96>(a, p, st);
        case 128: return dq_ordered_t<float, 128>(a, p, st);
        case 256: return dq_ordered_t<float, 256>(a, p, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace fa
