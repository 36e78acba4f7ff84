// packed_bwd_d256.cu -- attention backward over packed sequences at head dim 256, f16 / bf16, on
// the 5th-generation tensor cores.
//
//   S    = Q K^T            P    = exp2(S * scale*log2e - LSE*log2e)
//   dP   = dO V^T           dS   = P * (dP - D)
//   dV^T += dO^T P          dK^T += Q^T dS          dQacc += dS K  (fp32 reduction)
// The pipeline and the TMEM and shared-memory layout are those of the dense kernel of this head
// dim (bwd_d256.cu): 64-key CTAs, 64-row query tiles, dK and dV accumulated transposed.  As in
// packed_bwd.cu the key tiles come from the plan (a plan tile is two CTAs' keys), a long tile's
// iterations may be cut over several CTAs, Q, dO, K and V are read through tensor maps of the
// one sequence, and dS is formed from the unrounded P.  Bound like the dense kernel by the
// latency of its 64 x 64 tiles and the fp32 reductions of dQ: 2 x 4096 tokens, H = 16, H_kv = 4,
// causal bf16, 1490 us a call (460 TFLOP/s).
#include <math.h>

#include "bounded_wait.cuh"
#include "packed.cuh"

namespace fa {
namespace {

constexpr int D = 256;
constexpr int BM = 64;  // query rows per iteration
constexpr int BN = 64;  // key rows per CTA
constexpr int STAGES = 2;
constexpr int kPieces = kBwdTile / BN;  // CTAs per plan tile and head
constexpr int kThreads = 14 * 32;
constexpr int kWarpDrain0 = 0, kWarpSoft0 = 4, kNumSoftWarps = 8, kWarpTma = 12, kWarpMma = 13;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t TM_DV = 0, TM_DK = 128, TM_S = 256, TM_DP = 320, TM_DQ = 384;

constexpr uint32_t kBox = 64 * 128;                 // one 64-column box of a 64-row tile (8 KB)
constexpr uint32_t kTile = 4 * kBox;                // a 64 x 256 16-bit tile (32 KB)
constexpr uint32_t kPT = BM * 128;                  // a P or dS tile: 64 queries x 64 keys, 16-bit
constexpr uint32_t OFF_K = 0;
constexpr uint32_t OFF_V = OFF_K + kTile;
constexpr uint32_t OFF_Q = OFF_V + kTile;
constexpr uint32_t OFF_DO = OFF_Q + STAGES * kTile;
constexpr uint32_t OFF_P = OFF_DO + STAGES * kTile;
constexpr uint32_t OFF_DS = OFF_P + 2 * kPT;
constexpr uint32_t OFF_LSE = OFF_DS + 2 * kPT;
constexpr uint32_t OFF_DD = OFF_LSE + STAGES * BM * 4;
constexpr uint32_t OFF_BAR = OFF_DD + STAGES * BM * 4;

// Barrier slots.
enum {
    B_KV = 0,    // K, V landed (TMA)
    B_S_FULL,    // S(i) in TMEM (MMA commit)
    B_DP_FULL,   // dP(i) in TMEM (MMA commit)
    B_P_READY,   // P(i) in its shared tile, S read out of TMEM (8 softmax warps)
    B_DS_READY,  // dS(i) in its shared tile, dP read out of TMEM (8 softmax warps)
    B_DQ_FULL,   // a dQ half in TMEM (MMA commit; two phases per iteration)
    B_DQ_EMPTY,  // that half read out of TMEM (4 drain warps)
    B_PT_FREE,   // P tile k no longer read (MMA commit after the dV^T product); 2 slots
    B_DT_FREE = B_PT_FREE + 2,  // dS tile k no longer read (commit after the dQ products); 2 slots
    B_ACC = B_DT_FREE + 2,       // every product done (MMA commit)
    B_FINAL,     // MMA shutdown
    B_STAGE0     // STAGES "full" barriers, then STAGES "empty" barriers
};
constexpr uint32_t kNumBars = B_STAGE0 + 2 * STAGES;
constexpr uint32_t OFF_MISC = OFF_BAR + kNumBars * 8;
constexpr uint32_t SMEM = OFF_MISC + 16;
static_assert(SMEM <= 232448, "shared memory budget");

struct Params {
    PackedBwd a;
    BwdPlan plan;
    float scale_log2;
};

template <bool kBF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if (kBF16) {
        __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<uint32_t*>(&v);
    }
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

// 16 TMEM lanes x 32 columns starting at taddr (lane field = the quadrant's first lane):
// register 4j + 0/1 of thread t holds row t/4, columns 8j + 2(t%4) + 0/1; registers
// 4j + 2/3 hold row t/4 + 8, the same columns.
__device__ __forceinline__ void tmem_ld16x256_x4(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// 16 TMEM lanes x 128 columns: register 4j + 0/1 of thread t holds row t/4, columns
// 8j + 2(t%4) + 0/1; registers 4j + 2/3 row t/4 + 8 (j = 0..15).
__device__ __forceinline__ void tmem_ld16x256_x16(uint32_t taddr, uint32_t (&r)[64]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
        "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
        "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
          "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
          "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
          "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(taddr));
}

// Byte offset of element (row, col) of a 128-byte-swizzled tile with 128-byte rows
// (64 16-bit or 32 fp32 columns): 8-row atoms of 1024 bytes, 16-byte chunks XOR row % 8.
__device__ __forceinline__ uint32_t sw128_off(int row, int byte_in_row) {
    return (uint32_t)((row >> 3) * 1024 + (row & 7) * 128 + ((((byte_in_row >> 4) ^ (row & 7))) << 4) +
                      (byte_in_row & 15));
}

// dV and scale * dK for keys j0 .. j0 + 31 of the CTA's at head-dim index dcol, or their raw sums
// where the tile is cut
template <typename T>
__device__ __forceinline__ void write_dkv(const PackedBwd& a, long long k_tok, int hk, int rows, int j0, int dcol,
                                          float* part, const uint32_t (&rv)[32], const uint32_t (&rk)[32]) {
    T* dVb = static_cast<T*>(a.dV) + (k_tok + j0) * a.sdv.tok + hk * a.sdv.head + dcol;
    T* dKb = static_cast<T*>(a.dK) + (k_tok + j0) * a.sdk.tok + hk * a.sdk.head + dcol;
#pragma unroll
    for (int k = 0; k < 32; ++k) {
        if (j0 + k >= rows) continue;
        if (part != nullptr) {
            part[(j0 + k) * D + dcol] = __uint_as_float(rv[k]);
            part[(kBwdTile + j0 + k) * D + dcol] = __uint_as_float(rk[k]);
        } else {
            dVb[k * a.sdv.tok] = TypeTraits<T>::from_f32(__uint_as_float(rv[k]));
            dKb[k * a.sdk.tok] = TypeTraits<T>::from_f32(__uint_as_float(rk[k]) * a.scale);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    packed_bwd_d256_kernel(const __grid_constant__ Params p) {
    constexpr bool kBF16 = TypeTraits<T>::kId == FA_BF16;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = ptx::smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_MISC + 4);
    auto bar = [&](int i) { return sbase + OFF_BAR + 8u * (uint32_t)i; };
    auto bar_full = [&](int s) { return bar(B_STAGE0 + s); };
    auto bar_empty = [&](int s) { return bar(B_STAGE0 + STAGES + s); };

    ptx::griddep_launch_dependents();
    ptx::griddep_wait();  // the plan, D and the LSE copy
    const PackedBwd& a = p.a;
    unsigned int* const err = a.err;
    const bool skip_dq = a.deterministic != 0;  // a kernel of its own sums dQ in key order
    // ---- the CTA's 64 keys: a half of a plan tile; CTAs past the plan's end leave at once
    const int item = (int)blockIdx.x / kPieces, sub = (int)blockIdx.x % kPieces * BN;
    if (item / a.H_kv >= p.plan.head[1]) return;
    const KeyWork work = p.plan.work[item / a.H_kv];
    const KeyTile kt = p.plan.key[work.tile];
    const int hk = item % a.H_kv, g = a.H / a.H_kv;
    const int n0 = kt.n0 + sub, S_q = kt.S_q, S_k = kt.S_k;
    if (n0 >= S_k) return;
    const int off = S_k - S_q;  // query i sits at key position i + off
    Shape sh;
    sh.S_q = S_q;
    sh.S_k = S_k;
    sh.causal = a.causal;
    sh.window = a.window;
    int q_lo, q_hi;
    query_range(sh, n0, min(n0 + BN, S_k), q_lo, q_hi);
    const int m_start = q_lo / BM;
    const int m_end = q_hi > q_lo ? (q_hi + BM - 1) / BM : m_start;
    // this CTA's iterations it0 .. it0 + n_it - 1 of the tile's (all of them unless it is cut)
    const int all_it = g * (m_end - m_start);
    const int it0 = (int)((long long)all_it * work.part / work.parts);
    const int n_it = (int)((long long)all_it * (work.part + 1) / work.parts) - it0;
    auto iter_coords = [&](int it, int& h, int& m0) {
        m0 = (m_end - 1 - (it0 + it) / g) * BM;
        h = hk * g + (it0 + it) % g;
    };
    const long long row0 = (long long)kt.unit0 * kBwdTile;  // of the sequence in the padded rows
    // tensor maps of this sequence alone: rows past its ends read as zeros
    const CUtensorMap* tmQ = p.plan.maps + (size_t)kt.n * kSeqMaps;
    const CUtensorMap *tmdO = tmQ + 1, *tmK = tmQ + 2, *tmV = tmQ + 3;

    if (threadIdx.x == 0) {
        if ((sbase & 1023u) != 0) atomicOr(err, kErrSmemAlign);
        *abort_flag = (sbase & 1023u) != 0;
        for (int i = 0; i < (int)kNumBars; ++i) {
            uint32_t count = 1;
            if (i == B_P_READY || i == B_DS_READY) count = kNumSoftWarps;
            if (i == B_DQ_EMPTY) count = 4;
            ptx::mbar_init(bar(i), count);
        }
        ptx::fence_mbar_init();
        ptx::fence_proxy_async_smem();
    }
    if (warp == kWarpMma) {
        ptx::tmem_alloc(sbase + OFF_MISC + 4, kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == kWarpTma) {
        // ------------------------------------------------------------ producer
        if (lane == 0 && !*abort_flag) {
            for (int i = 0; i < 4; ++i) tensormap_acquire(tmQ + i);  // written by the plan kernel
            ptx::fence_proxy_async_global();  // the LSE copy and D, written by the preprocess pass
            ptx::mbar_arrive_expect_tx(bar(B_KV), 2 * kTile);
            for (int x = 0; x < 4; ++x) {
                ptx::tma_load_3d(sbase + OFF_K + x * kBox, tmK, x * 64, hk, n0, bar(B_KV));
                ptx::tma_load_3d(sbase + OFF_V + x * kBox, tmV, x * 64, hk, n0, bar(B_KV));
            }
            auto load_stage = [&](int it) {
                const int s = it % STAGES;
                int h, m0;
                iter_coords(it, h, m0);
                ptx::mbar_arrive_expect_tx(bar_full(s), 2 * kTile + 2 * BM * 4);
                for (int x = 0; x < 4; ++x) {
                    ptx::tma_load_3d(sbase + OFF_Q + s * kTile + x * kBox, tmQ, x * 64, h, m0, bar_full(s));
                    ptx::tma_load_3d(sbase + OFF_DO + s * kTile + x * kBox, tmdO, x * 64, h, m0, bar_full(s));
                }
                const size_t row = (size_t)(h * p.plan.rows + row0 + m0);
                ptx::bulk_load(sbase + OFF_LSE + s * BM * 4, p.plan.lse2 + row, BM * 4, bar_full(s));
                ptx::bulk_load(sbase + OFF_DD + s * BM * 4, p.plan.D + row, BM * 4, bar_full(s));
            };
            int issued = 0;
            for (int it = 0; it < n_it; ++it) {
                const int s = it % STAGES;
                // stage s was last read by the dK^T product of iteration it - 2 (MMA commit)
                if (it >= STAGES && !wait_bar(bar_empty(s), ((it / STAGES) - 1) & 1, abort_flag, err)) break;
                load_stage(it);
                issued = it + 1;
            }
            // never leave copies in flight into shared memory that is about to be released
            drain_wait(bar(B_KV), 0);
            for (int it = issued - STAGES < 0 ? 0 : issued - STAGES; it < issued; ++it)
                drain_wait(bar_full(it % STAGES), (it / STAGES) & 1);
        }
    } else if (warp == kWarpMma) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0 && !*abort_flag && n_it > 0) {
            constexpr uint32_t ID_S = ptx::idesc_f16(64, 64, kBF16, false, false);   // S, dP
            constexpr uint32_t ID_T = ptx::idesc_f16(128, 64, kBF16, true, true);    // dV^T, dK^T
            constexpr uint32_t ID_Q = ptx::idesc_f16(64, 128, kBF16, false, true);   // dQ halves
            const uint32_t sK = sbase + OFF_K, sV = sbase + OFF_V;
            // S = Q K^T or dP = dO V^T (M = 64 queries, N = 64 keys, 16 K-steps over d; both
            // operands K-major)
            auto gemm_s = [&](uint32_t d_tmem, uint32_t a_base, uint32_t b_base) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t koff = (k / 4) * kBox + (k % 4) * 32;
                    ptx::mma_ss(d_tmem, ptx::sw128_desc(a_base + koff, 16, 1024),
                                ptx::sw128_desc(b_base + koff, 16, 1024), ID_S, k > 0);
                }
            };
            // acc^T += X^T Y for the two 128-row halves of d: A = X^T (MN-major: the 16-bit
            // [64 x 256] tile, two 64-column boxes per half), B = Y (the [64 x 64] P or dS
            // tile, MN-major); K = the 64 queries in 4 steps
            auto gemm_t = [&](uint32_t d_tmem, uint32_t x_base, uint32_t y_base, bool acc) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int k = 0; k < BM / 16; ++k)
                        ptx::mma_ss(d_tmem + 64 * h, ptx::sw128_desc(x_base + 2 * h * kBox + k * 2048, kBox, 1024),
                                    ptx::sw128_desc(y_base + k * 2048, kPT, 1024), ID_T, (acc || k > 0) ? 1u : 0u);
            };
            // dQ half h = dS K[:, 128h, 128h + 128): A = dS (K-major over the 64 keys), B = K
            // (MN-major, two 64-column boxes)
            auto gemm_q = [&](uint32_t ds_base, int h) {
#pragma unroll
                for (int k = 0; k < BN / 16; ++k)
                    ptx::mma_ss(tmem + TM_DQ, ptx::sw128_desc(ds_base + k * 32, 16, 1024),
                                ptx::sw128_desc(sK + 2 * h * kBox + k * 2048, kBox, 1024), ID_Q, k > 0);
            };
            bool ok = wait_bar(bar(B_KV), 0, abort_flag, err);
            if (ok) ok = wait_bar(bar_full(0), 0, abort_flag, err);
            if (ok) {
                ptx::tc_fence_after();
                gemm_s(tmem + TM_S, sbase + OFF_Q, sK);
                ptx::mma_commit(bar(B_S_FULL));
                gemm_s(tmem + TM_DP, sbase + OFF_DO, sV);
                ptx::mma_commit(bar(B_DP_FULL));
            }
            for (int it = 0; ok && it < n_it; ++it) {
                const int s = it % STAGES, s1 = (it + 1) % STAGES;
                const uint32_t sQ = sbase + OFF_Q + s * kTile, sdO = sbase + OFF_DO + s * kTile;
                const uint32_t sP = sbase + OFF_P + (it & 1) * kPT, sdS = sbase + OFF_DS + (it & 1) * kPT;
                // dV^T += dO^T P once P(i) is in its tile (the softmax read S(i) before)
                if (!(ok = wait_bar(bar(B_P_READY), it & 1, abort_flag, err))) break;
                ptx::tc_fence_after();
                gemm_t(tmem + TM_DV, sdO, sP, it > 0);
                ptx::mma_commit(bar(B_PT_FREE + (it & 1)));
                // S(i+1) into the S buffer (read out already)
                if (it + 1 < n_it) {
                    if (!(ok = wait_bar(bar_full(s1), ((it + 1) / STAGES) & 1, abort_flag, err))) break;
                    ptx::tc_fence_after();
                    gemm_s(tmem + TM_S, sbase + OFF_Q + s1 * kTile, sK);
                    ptx::mma_commit(bar(B_S_FULL));
                }
                // dK^T += Q^T dS once dS(i) is in its tile (the softmax read dP(i) before)
                if (!(ok = wait_bar(bar(B_DS_READY), it & 1, abort_flag, err))) break;
                ptx::tc_fence_after();
                gemm_t(tmem + TM_DK, sQ, sdS, it > 0);
                ptx::mma_commit(bar_empty(s));  // Q(i), dO(i) read for the last time
                if (!skip_dq) {
                    // dQ low half into the dQ buffer once the drain read the previous high half
                    if (it > 0 && !(ok = wait_bar(bar(B_DQ_EMPTY), 1, abort_flag, err))) break;
                    ptx::tc_fence_after();
                    gemm_q(sdS, 0);
                    ptx::mma_commit(bar(B_DQ_FULL));
                }
                // dP(i+1) while the drain reads the low half (the dP buffer was read out already)
                if (it + 1 < n_it) {
                    gemm_s(tmem + TM_DP, sbase + OFF_DO + s1 * kTile, sV);
                    ptx::mma_commit(bar(B_DP_FULL));
                }
                if (!skip_dq) {
                    if (!(ok = wait_bar(bar(B_DQ_EMPTY), 0, abort_flag, err))) break;
                    ptx::tc_fence_after();
                    gemm_q(sdS, 1);
                    ptx::mma_commit(bar(B_DQ_FULL));
                }
                ptx::mma_commit(bar(B_DT_FREE + (it & 1)));
            }
            ptx::mma_commit(bar(B_ACC));
            // no MMA may still write TMEM when it is released
            ptx::mma_commit(bar(B_FINAL));
            drain_wait(bar(B_FINAL), 0);
        }
        __syncwarp();
    } else if (warp >= kWarpSoft0 && warp < kWarpSoft0 + kNumSoftWarps) {
        // ------------------------------------------------------------ P / dS
        // Warp (quadrant qd, key half hc): query rows 16 qd + t/4 and 16 qd + t/4 + 8 of the
        // tile, keys 32 hc + 8j + 2(t%4) + 0/1 (j = 0..3), from TMEM lanes 32 qd ...
        const int qd = warp & 3;
        const int hc = (warp - kWarpSoft0) >> 2;
        const uint32_t lane_base = (uint32_t)(qd * 32) << 16;
        const int ra = 16 * qd + (lane >> 2), rb = ra + 8;  // the thread's two query rows
        const int c0 = 32 * hc + 2 * (lane & 3);             // its first key column
        bool ok = !*abort_flag;
        for (int it = 0; ok && it < n_it; ++it) {
            const int s = it % STAGES;
            int h, m0;
            iter_coords(it, h, m0);
            const float* sl = reinterpret_cast<const float*>(smem + OFF_LSE + s * BM * 4);
            const float* sd = reinterpret_cast<const float*>(smem + OFF_DD + s * BM * 4);
            // every element of the tile visible (no mask needed): the extreme query-key
            // offsets of the tile satisfy the causal and window conditions, no key past S_k
            const int pk_min = m0 + off - (n0 + BN - 1), pk_max = m0 + BM - 1 + off - n0;
            const bool full = n0 + BN <= S_k && (!a.causal || pk_min >= 0) &&
                              (a.window <= 0 || (pk_max < a.window && (a.causal || -pk_min < a.window)));
            if (!(ok = wait_bar_warp(bar_full(s), (it / STAGES) & 1, abort_flag, err))) break;
            if (!(ok = wait_bar_warp(bar(B_S_FULL), it & 1, abort_flag, err))) break;
            ptx::tc_fence_after();
            uint32_t r[16];
            tmem_ld16x256_x4(tmem + TM_S + lane_base + 32 * hc, r);
            ptx::tmem_wait_ld();
            const float la = sl[ra], lb = sl[rb];
            float pv[16];  // P at (row, col) in the register layout of r
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int row = (e & 2) ? rb : ra;
                const int col = c0 + 8 * (e >> 2) + (e & 1);
                float x = ptx::ex2(fmaf(__uint_as_float(r[e]), p.scale_log2, -((e & 2) ? lb : la)));
                if (!full) {
                    const int j = n0 + col;
                    x = (j < S_k && key_visible(m0 + row + off, j, a.causal, a.window)) ? x : 0.f;
                }
                pv[e] = x;
            }
            // the P tile of this parity was last read by the dV^T product two iterations ago
            if (it >= 2 && !(ok = wait_bar_warp(bar(B_PT_FREE + (it & 1)), ((it >> 1) - 1) & 1, abort_flag, err)))
                break;
            uint8_t* tP = smem + OFF_P + (it & 1) * kPT;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int cb = 2 * (c0 + 8 * j);  // byte of the column pair within the row
                *reinterpret_cast<uint32_t*>(tP + sw128_off(ra, cb)) = pack2<kBF16>(pv[4 * j], pv[4 * j + 1]);
                *reinterpret_cast<uint32_t*>(tP + sw128_off(rb, cb)) = pack2<kBF16>(pv[4 * j + 2], pv[4 * j + 3]);
            }
            ptx::tc_fence_before();
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(B_P_READY));

            // dS = P * (dP - D)
            if (!(ok = wait_bar_warp(bar(B_DP_FULL), it & 1, abort_flag, err))) break;
            if (it >= 2 && !(ok = wait_bar_warp(bar(B_DT_FREE + (it & 1)), ((it >> 1) - 1) & 1, abort_flag, err)))
                break;
            ptx::tc_fence_after();
            tmem_ld16x256_x4(tmem + TM_DP + lane_base + 32 * hc, r);
            ptx::tmem_wait_ld();
            const float da = sd[ra], db = sd[rb];
            uint8_t* tS = smem + OFF_DS + (it & 1) * kPT;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float ds[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int e = 4 * j + u;
                    ds[u] = pv[e] * (__uint_as_float(r[e]) - ((u & 2) ? db : da));
                }
                const int cb = 2 * (c0 + 8 * j);
                *reinterpret_cast<uint32_t*>(tS + sw128_off(ra, cb)) = pack2<kBF16>(ds[0], ds[1]);
                *reinterpret_cast<uint32_t*>(tS + sw128_off(rb, cb)) = pack2<kBF16>(ds[2], ds[3]);
            }
            ptx::tc_fence_before();
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar(B_DS_READY));
        }
        // ---- epilogue: dV^T and scale * dK^T rows (one head-dim index per thread) to dV, dK, or a
        // part's sums to its slot
        if (ok && n_it > 0) ok = wait_bar_warp(bar(B_ACC), 0, abort_flag, err);
        if (ok) {
            float* part = work.parts > 1 ? p.plan.part + (((size_t)work.slot * a.H_kv + hk) * 2 * kBwdTile + sub) * D : nullptr;
            ptx::tc_fence_after();
            const int dcol = 128 * hc + 32 * qd + lane;  // head-dim index of this thread
#pragma unroll
            for (int c = 0; c < BN / 32; ++c) {
                uint32_t rv[32], rk[32];
                if (n_it > 0) {
                    ptx::tmem_ld32p(tmem + TM_DV + 64 * hc + lane_base + 32 * c, rv);
                    ptx::tmem_ld32p(tmem + TM_DK + 64 * hc + lane_base + 32 * c, rk);
                    ptx::tmem_wait_ld();
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) rv[k] = rk[k] = 0u;
                }
                write_dkv<T>(a, kt.k_tok + sub, hk, min(BN, S_k - n0), 32 * c, dcol, part, rv, rk);
            }
        }
    } else if (warp >= kWarpDrain0 && warp < kWarpDrain0 + 4) {
        // ------------------------------------------------------------ dQ drain
        // Warp qd reads the 16 query rows of its lane quadrant, a whole 128-column half at a
        // time, with all 32 threads (rows t/4 and t/4 + 8, column pairs), releases the TMEM
        // buffer, then adds the values into the accumulator rows with fp32 vector reductions.
        const int qd = warp;
        const uint32_t lane_base = (uint32_t)(qd * 32) << 16;
        const int ra = 16 * qd + (lane >> 2), rb = ra + 8;
        const int c0 = 2 * (lane & 3);
        float* const acc = p.plan.dqacc + ((long long)kt.q_tok + ra) * a.H * D + c0;  // the thread's first row
        bool ok = !*abort_flag && !skip_dq;
        for (int it = 0; ok && it < n_it; ++it) {
            int h, m0;
            iter_coords(it, h, m0);
            const bool a_ok = m0 + ra < S_q, b_ok = m0 + rb < S_q;
            float* ga = acc + ((long long)m0 * a.H + h) * D;
            float* gb = ga + 8ll * a.H * D;
#pragma unroll 1
            for (int hc = 0; hc < 2; ++hc) {
                if (!(ok = wait_bar_warp(bar(B_DQ_FULL), hc, abort_flag, err))) break;
                ptx::tc_fence_after();
                uint32_t r[64];
                tmem_ld16x256_x16(tmem + TM_DQ + lane_base, r);
                ptx::tmem_wait_ld();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(B_DQ_EMPTY));
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int col = 128 * hc + 8 * j;
                    if (a_ok) ptx::red_add_v2(ga + col, __uint_as_float(r[4 * j]), __uint_as_float(r[4 * j + 1]));
                    if (b_ok) ptx::red_add_v2(gb + col, __uint_as_float(r[4 * j + 2]), __uint_as_float(r[4 * j + 3]));
                }
            }
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == kWarpMma) ptx::tmem_dealloc(tmem, kTmemCols);
}

template <typename T>
cudaError_t launch_t(const PackedBwd& a, const BwdPlan& plan, cudaStream_t st) {
    if (plan.max_keys == 0) return cudaSuccess;  // no key rows
    Params p;
    p.a = a;
    p.plan = plan;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    auto kern = packed_bwd_d256_kernel<T>;
    static std::atomic<uint64_t> ready{0};
    cudaError_t e = allow_smem(kern, (int)SMEM, ready);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long long)plan.max_work * a.H_kv * kPieces));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_packed_bwd_d256(const PackedBwd& a, const BwdPlan& p, cudaStream_t st) {
    return a.dtype == FA_F16 ? launch_t<__half>(a, p, st) : launch_t<__nv_bfloat16>(a, p, st);
}

}  // namespace fa
