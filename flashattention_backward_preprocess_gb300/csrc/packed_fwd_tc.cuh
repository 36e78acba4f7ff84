// packed_fwd_tc.cuh -- attention forward over packed sequences or a paged key/value cache for
// GB300 (sm_103a), f16 / bf16, on the 5th-generation tensor cores.
//
//   s_ij = scale <q_i, k_j> over the keys j of i's own sequence that it sees (key_visible)
//   O_i  = sum_j exp(s_ij) v_j / sum_j exp(s_ij),   LSE_i = log sum_j exp(s_ij)
// with one pass over the keys (running max and sum per row); a row that sees no key gets
// O = 0 and LSE = -inf.
//
// Design:
//   * a tile packs tpt = 128 / g query tokens with the g query heads of one key/value head
//     (one TMA box [64 columns, g heads, tpt tokens]), so keys and values are read once per
//     group: a single-token step reads its cache once, whatever the number of query heads;
//   * the plan kernel lays all (unit, key/value head, key tile) triples on one axis and gives
//     each of the CTAs (one per SM) the same number of them.  One long request is spread over
//     the whole grid by the same rule that packs a thousand short ones.  Items that a share's
//     border cuts leave fp32 parts in the workspace; the CTA whose part arrives last joins
//     them in order of the keys, so the result does not depend on which one that is;
//   * K / V tiles come through a TMA ring.  Paged: one box per page, 128-byte swizzle, each
//     lane of the producer warp looks up and issues its own boxes one tile ahead.  The rows of
//     V behind the sequence's last key (another sequence's, or whatever a page holds) are
//     zeroed in shared memory before the P V product: P is 0 there, but 0 * inf is not;
//   * S = Q K^T and O += P V with tcgen05.mma, P as the TMEM A operand; three S buffers
//     (two at d = 256); eight softmax warps (two threads per row), four epilogue warps, a warp
//     each for the loads of Q and K, the loads of V, the S products and the P V products.  The
//     next item's loads, S products and softmax overlap this item's epilogue.  Softmax warps
//     whose rows are all padding (single-token steps fill g of 128 rows) only pass the
//     barriers on;
//   * P is rounded to the inputs' 16-bit type for the product (the tensor core's operand type);
//     the row sum adds the unrounded fp32 values;
//   * every wait is bounded: a timeout records an error word, the roles drop out, TMEM is freed.
//
// Bound by the softmax on long prompts (about 1250 cycles of a key tile's 1400) and nearly as much by
// the products (1310 from the first to the last of a tile, in which the tensor pipe itself is active
// 53 to 60 % of the time: it waits for operands too), by DRAM on single-token steps, by latency on
// small calls.  Measured, causal bf16, times of a replayed graph: 4 x 4096 tokens, H = 32, H_kv =
// 8, d = 128 401 us (1370 TFLOP/s), 8 prompts of 1 to 4096 tokens (16280 in all) 333 us (1220
// TFLOP/s); 4 x 4096, H = H_kv = 16, d = 64 195 us (705 TFLOP/s); 2 x 4096, H = 16, H_kv = 4,
// d = 256 274 us (1000 TFLOP/s); 64 requests, one token each, over 1.14 GB of a cache of 16-row
// pages 178 us (6.4 TB/s).
#pragma once

#include <math.h>

#include "bounded_wait.cuh"
#include "packed.cuh"
#include "packed_q8.cuh"
#include "tma_map.cuh"

namespace fa {
namespace {

constexpr int BM = 128;  // rows per tile
// warps 0-7 softmax, 8-11 epilogue, 12 loads of Q and K, 13 S products and TMEM, 14 P V products,
// 15 loads of V
// 8-bit caches: 12 and 15 look rows of K and V up, 16-23 load and convert them, 13 loads Q as well
constexpr int kWarpEpi = 8, kWarpLoadK = 12, kWarpMma = 13, kWarpPv = 14, kWarpLoadV = 15, kWarpConv = 16;
constexpr uint32_t kTmemCols = 512;
constexpr float kMaxSum = 16384.f;    // of a tile's half row before the running max is looked at again
// 8-bit caches: P is fp16 whatever Q's type, so it is kept 2^8 above the reference: its fixed step
// below 2^-14 is 2^-33 of the largest P then (for bf16 queries 2^-25 would show)
constexpr float kQ8Lift = 8.f, kQ8MaxSum = 57344.f;
constexpr uint32_t kEpiBarrier = 1;   // the epilogue's four warps
constexpr uint32_t kPairBarrier = 2;  // + lane quadrant: the two softmax warps of a row

template <int D, bool kQ8>
struct PCfg {
    static constexpr int THREADS = kQ8 ? 768 : 512;
    // registers per thread of the two softmax warpgroups, the epilogue, the last one and the two
    // converting ones: together what the block is launched with, 4 x 128 or (65536 / 768, a whole
    // multiple of 8) 6 x 80
    static constexpr int REGS_SOFT = kQ8 ? 104 : 152, REGS_EPI = kQ8 ? 88 : 120, REGS_OTHER = kQ8 ? 56 : 88, REGS_CONV = 64;
    static constexpr int REGS = kQ8 ? 80 : 128;
    static_assert(2 * REGS_SOFT + REGS_EPI + REGS_OTHER + (kQ8 ? 2 * REGS_CONV : 0) == THREADS / 128 * REGS, "see above");
    static_assert(REGS_SOFT >= REGS && REGS_OTHER <= REGS && REGS_CONV <= REGS, "raised or lowered as the roles do");
    static constexpr int BN = D <= 128 ? 128 : 64;
    // slots of the K and of the V ring
    static constexpr int KST = kQ8 ? (D == 64 ? 3 : 2) : (D == 64 ? 4 : (D == 128 ? 3 : 2));
    static constexpr int VST = KST;
    static constexpr int INFO = kQ8 ? 4 : 0;  // slots of the ring of looked-up tiles
    static constexpr int NBUF = D <= 128 ? 3 : 2;
    static constexpr int BOXES = D / 64;
    static constexpr uint32_t kTileQ_B = BM * D * 2;
    static constexpr uint32_t kTileKV_B = BN * D * 2;
    static constexpr uint32_t kBoxQ_B = BM * 128;
    static constexpr uint32_t kBoxKV_B = BN * 128;
    static constexpr uint32_t OFF_Q = 0;
    static constexpr uint32_t OFF_K = OFF_Q + kTileQ_B;
    static constexpr uint32_t OFF_V = OFF_K + KST * kTileKV_B;
    // float2 per row: two slots of the rows' max and sum; then a float per row that a row's two
    // softmax threads exchange
    static constexpr uint32_t OFF_ROW = OFF_V + VST * kTileKV_B;
    static constexpr uint32_t OFF_XCH = OFF_ROW + 2 * BM * 8;
    // 8-bit caches.  Of a looked-up tile: where its rows lie in K and in V, their exponents, words of
    // both halves; for the softmax its largest exponents and, where they are needed, all of them (8 slots
    // each); of an item's rows: the inverse of the power of two that Q was scaled by (4 slots)
    static constexpr uint32_t OFF_AT = OFF_XCH + BM * 4;
    static constexpr uint32_t OFF_EXP = OFF_AT + INFO * BN * 16;
    static constexpr uint32_t OFF_INFO = OFF_EXP + INFO * BN * 2;
    static constexpr uint32_t OFF_TOP = OFF_INFO + INFO * 16;
    static constexpr uint32_t OFF_QS = OFF_TOP + (kQ8 ? 32 : 0);
    static constexpr uint32_t OFF_FAR = OFF_QS + (kQ8 ? 4 * BM * 4 : 0);
    static constexpr uint32_t OFF_BAR = OFF_FAR + (kQ8 ? 8 * BN * 2 : 0);
    // V(j)'s slot is past V(j - VST) once S(j) is complete (the softmax warps' rare waits for V)
    static_assert(kQ8 || VST >= NBUF, "see above");
    // what the softmax reads of a tile's or item's slot is read before the slot is written again
    static_assert(!kQ8 || KST + NBUF < 8, "see above");
    static_assert(OFF_AT % 16 == 0 && OFF_INFO % 8 == 0 && OFF_FAR % 16 == 0 && OFF_BAR % 8 == 0, "alignment");
    static constexpr uint32_t TM_S = 0, TM_O = 128 * NBUF;
    static_assert(TM_O + D <= 512, "TMEM columns");
};

enum {
    P_Q = 0,               // Q tile landed (TMA)
    P_S0,                  // S in buffer b (MMA commit), three slots
    P_P0 = P_S0 + 3,       // P packed in buffer b (8 softmax warps), three slots
    P_PV0 = P_P0 + 3,      // P V product of buffer b done (MMA commit), three slots
    P_FINAL = P_PV0 + 3,   // every product done
    P_QE,                  // the item's S products are done: the Q tile may be reloaded
    P_OFULL,               // O of an item complete
    P_OFREE,               // O of an item read (4 epilogue warps)
    P_ML0,                 // max and sum of an item's rows written (4 softmax warps), 2 slots
    P_MR0 = P_ML0 + 2,     // and read by the epilogue (4 warps), 2 slots
    P_SLOT0 = P_MR0 + 2    // KST "full" and KST "empty" of the K ring, VST of each of the V ring, and
                           // for 8-bit caches Q made fp16 (4 converting warps), then INFO "full" and
                           // INFO "empty" of the ring of looked-up tiles
};

// 8-bit caches: arrivals at barrier P_SLOT0 + i.  Four converting warps make K (and Q), four V, all
// eight free the looked-up tiles, which two warps look up.
template <typename C>
__device__ __forceinline__ uint32_t q8_arrivals(int i) {
    constexpr int q = 2 * (C::KST + C::VST);
    if (i > q) return i <= q + C::INFO ? 2u : 8u;
    return i < C::KST || (i >= 2 * C::KST && i < 2 * C::KST + C::VST) || i == q ? 4u : 1u;
}

__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// TMEM column (relative to a buffer) of the packed 16-bit P for 16 keys, MMA k-step k: each half
// of the BN key columns is packed into the first half of the columns it was read from.
template <int BN>
__device__ __forceinline__ constexpr uint32_t packed_col(int k) {
    return (uint32_t)((k / (BN / 32)) * (BN / 2) + (k % (BN / 32)) * 8);
}
// Bits k0 .. k0 + n - 1 of a token's mask (`words` 64-bit words; set below 0: the tokens before the
// new ones, clear behind the last word).
template <int n>
__device__ __forceinline__ unsigned long long tree_columns(const unsigned long long* mask, int words, int k0) {
    if (k0 + n <= 0) return ~0ull;
    if (k0 < 0) return (mask[0] << -k0) | ((1ull << -k0) - 1ull);
    const int w = k0 >> 6, s = k0 & 63;
    const unsigned long long lo = w < words ? mask[w] : 0ull, hi = s + n > 64 && w + 1 < words ? mask[w + 1] : 0ull;
    return s ? (lo >> s) | (hi << (64 - s)) : lo;
}
template <bool kBF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if (kBF16) {
        __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<uint32_t*>(&v);
    }
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* map, int c0, int c1, int c2) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(c2)
                 : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
        : "memory");
}

// A thread's N scores of a far tile (packed_q8.cuh), in TMEM from `buf` on: the operands hold K's and V's numbers
// as they are, so a key's own exponents go to its score and to its P.  exps: the keys' exponent bytes, K's in
// the low ones.
// Scores s to y = scale 2^ek s + ev, -inf in the columns without see(column); returns the largest.
template <int N, typename See>
__device__ __forceinline__ float far_scores(uint32_t buf, const uint16_t* exps, float scale, See see) {
    float most = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < N; c += 32) {
        uint32_t y[32];
        ptx::tmem_ld32p(buf + c, y);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const uint32_t e = exps[c + i];
            const float ev = (float)((int)max(e >> 8, kMinExp) - 127);
            const float x = fmaf(__uint_as_float(y[i]), scale * __uint_as_float((e & 0xff) << 23), ev);
            y[i] = __float_as_uint(see(c + i) ? x : -INFINITY);
            most = fmaxf(most, __uint_as_float(y[i]));
        }
        ptx::tmem_st32(buf + c, y);
    }
    ptx::tmem_wait_st();
    return most;
}
// y to P 2^ev = 2^(y - m), packed into the first half of the columns; returns the sum of P.
template <int N, bool kBF16>
__device__ __forceinline__ float far_weights(uint32_t buf, const uint16_t* exps, float m) {
    float sum = 0.f;
#pragma unroll 1
    for (int c = 0; c < N; c += 32) {
        uint32_t y[32], p[16];
        ptx::tmem_ld32p(buf + c, y);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            const float p0 = ptx::ex2(__uint_as_float(y[i]) - m), p1 = ptx::ex2(__uint_as_float(y[i + 1]) - m);
            sum = fmaf(p0, __uint_as_float((254u - max((uint32_t)exps[c + i] >> 8, kMinExp)) << 23), sum);
            sum = fmaf(p1, __uint_as_float((254u - max((uint32_t)exps[c + i + 1] >> 8, kMinExp)) << 23), sum);
            p[i / 2] = pack2<kBF16>(p0, p1);
        }
        ptx::tmem_st16(buf + c / 2, p);
    }
    return sum;
}

// 32 bytes per thread (32-byte aligned): a row per thread makes every store of a warp touch 32
// lines, so the widest store has the fewest of them
__device__ __forceinline__ void st_global_v8(void* p, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2, int c3,
                                            int c4, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
        : "memory");
}

// kPaged: K / V from a cache.  kGroup (paged, d a whole multiple of 64 and above 64): one box
// per page and tensor brings all its columns, so a tile lies in shared memory as groups of 8
// rows, each with its 64-column blocks one after another, instead of one block of all rows
// after another.  Small boxes are what bounds a cache of small pages (about 60 ns a box,
// whatever it holds): a step of 64 tokens over 4096 each in pages of 16 rows took 253 us with
// a box per 64 columns and 175 us with one per page.
// kTree (paged): new tokens see each other by the call's masks.  kQ8 (paged): an 8-bit cache
// (packed_q8.cuh), whose tiles the converting warps load.
template <typename T, int D, bool kPaged, bool kGroup, bool kTree, bool kQ8>
__global__ void __launch_bounds__(PCfg<D, kQ8>::THREADS, 1)
    packed_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const PackedFwd a, const FwdPlan plan, const FwdGeom geo, int max_units) {
    using C = PCfg<D, kQ8>;
    constexpr int BN = C::BN, NB = C::NBUF, kThreads = C::THREADS;
    // K / V tile layout: bytes from a 64-column block to the next, and from 8 rows to the next 8
    constexpr uint32_t kBlk = kGroup ? 1024 : C::kBoxKV_B;
    constexpr uint32_t kRow8 = kGroup ? 1024 * C::BOXES : 1024;
    constexpr int kPerPage = kGroup ? 1 : C::BOXES;          // boxes per page of K or V
    constexpr int kPieces = (BN / 8 * kPerPage + 31) / 32;  // and tile per producer lane (pages of 8 rows)
    constexpr bool kBF16 = TypeTraits<T>::kId == FA_BF16;
    constexpr bool kOpBF16 = kBF16 && !kQ8;  // operands of the products
    constexpr bool kConvQ = kBF16 && kQ8;    // Q is made fp16
    constexpr int kNumBars = P_SLOT0 + 2 * C::KST + 2 * C::VST + (kQ8 ? 1 + 2 * C::INFO : 0);
    constexpr uint32_t OFF_MISC = C::OFF_BAR + kNumBars * 8;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = ptx::smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_MISC + 4);
    volatile int* last_flag = reinterpret_cast<volatile int*>(smem + OFF_MISC + 8);
    auto bar = [&](int i) { return sbase + C::OFF_BAR + 8u * (uint32_t)i; };
    // a ring each for K and V: a K slot is free once S is computed, well before V's
    auto k_full = [&](int s) { return bar(P_SLOT0 + s); };
    auto k_empty = [&](int s) { return bar(P_SLOT0 + C::KST + s); };
    auto v_full = [&](int s) { return bar(P_SLOT0 + 2 * C::KST + s); };
    auto v_empty = [&](int s) { return bar(P_SLOT0 + 2 * C::KST + C::VST + s); };
    [[maybe_unused]] const uint32_t q_conv = bar(P_SLOT0 + 2 * C::KST + 2 * C::VST);
    [[maybe_unused]] const Q8Bars<C> q8_bars = {k_full(0), k_empty(0), v_full(0), v_empty(0), bar(P_Q), q_conv, q_conv + 8u};
    const int g = a.H / a.H_kv;
    unsigned int* err = a.err;

    if (threadIdx.x == 0) {
        if ((sbase & 1023u) != 0) atomicOr(err, kErrSmemAlign);
        *abort_flag = (sbase & 1023u) != 0;
        for (int i = 0; i < kNumBars; ++i)
            ptx::mbar_init(bar(i), i >= P_P0 && i < P_P0 + 3 ? 8u
                                   : i >= P_OFREE && i < P_SLOT0 ? 4u
                                   : kQ8 && i >= P_SLOT0 ? q8_arrivals<C>(i - P_SLOT0) : 1u);
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
    ptx::griddep_wait();  // the plan, or with it the lengths
    FwdShare share;
    if (geo.self) {
        SelfPlan* sp = reinterpret_cast<SelfPlan*>(smem + C::OFF_K);  // before any tile lands there
        plan_self<kThreads>(a, geo, plan, max_units, sp);
        share = sp->share;
        ptx::fence_proxy_async_smem();
        // without any work (lengths that do not fit, say) no row belongs to a sequence
        if (a.fill) fill_rows<T>(a, share.W == 0, blockIdx.x * kThreads + threadIdx.x, (long long)gridDim.x * kThreads);
        __syncthreads();
    } else {
        share.read(plan, blockIdx.x);
    }
    if (kPaged && a.gate != nullptr && __ldcg(a.gate) != a.gate_value) share.W = 0;  // another kernel's step

    // Every role walks the same segments.  Per-tile barrier phases count the key tiles of this
    // CTA (jg), per-item ones its segments with work (ka).
    if (kQ8 && warp >= kWarpConv) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_CONV));
        if constexpr (kQ8) {
            if (!*abort_flag) convert_tiles<C, D, kConvQ>(a, smem, abort_flag, q8_bars);
        }
    } else if (warp >= kWarpLoadK) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_OTHER));
    if (kQ8 && (warp == kWarpLoadK || warp == kWarpLoadV)) {
        // ------------------------------------------------------------ rows of K and V (8-bit caches)
        if constexpr (kQ8) {
            if (!*abort_flag) look_up_tiles<C>(a, share, geo, smem, abort_flag, q8_bars, warp == kWarpLoadV);
        }
        __syncwarp();
    } else
    if (warp == kWarpLoadK || warp == kWarpLoadV) {
        // ------------------------------------------------------------ producers
        // One warp loads the Q tile of each item (once the previous item's S products are done)
        // and its K tiles, the other the V tiles; every lane issues its own boxes of a tile.
        const bool is_v = warp == kWarpLoadV;
        const CUtensorMap* map = is_v ? &tmV : &tmK;
        const uint32_t ring = sbase + (is_v ? C::OFF_V : C::OFF_K);
        const int hs = (int)(is_v ? a.v.head : a.k.head);
        const int pr = kPaged ? min(a.page_size, BN) : BN;           // rows per box
        const int per_tile = BN / pr;                                // pages per tile
        const int tiles_page = kPaged ? max(a.page_size / BN, 1) : 1;  // or tiles per page
        int q_act = 0, jg = 0;  // Q tiles and ring tiles loaded
        // paged: table entries of this lane's boxes of the next tile.  They are only loaded here
        // and looked at when the tile is issued, so the load's latency passes meanwhile.
        int page[kPieces];
        int live = 0;  // boxes of that tile that hold a key
        FwdWalk w;
        bool ok = !*abort_flag;
        bool more = ok && w.init(share, blockIdx.x, a.H_kv, geo.overhead);
        while (more && w.tiles() == 0) more = w.next();
        int j = more ? w.j0 : 0;
        auto look_up = [&]() {
            if constexpr (kPaged) {
                const int tile = w.t.n_first + j;
                live = min((w.t.S_k - tile * BN + pr - 1) / pr, per_tile);
                const int* row = a.table + (size_t)w.t.n * a.max_pages;
                const int e0 = tiles_page > 1 ? tile / tiles_page : tile * per_tile;
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const int b = (lane + 32 * i) / kPerPage;
                    page[i] = b < live && e0 + b < a.max_pages ? row[e0 + b] : -1;
                }
            }
        };
        if (more) look_up();
        while (more) {
            if (!is_v && j == w.j0) {
                if (q_act > 0 && !(ok = wait_bar_warp(bar(P_QE), (q_act - 1) & 1, abort_flag, err))) break;
                if (lane == 0) ptx::mbar_arrive_expect_tx(bar(P_Q), (uint32_t)(geo.tpt * g) * 128u * C::BOXES);
                __syncwarp();
                if (lane < C::BOXES)
                    ptx::tma_load_3d(sbase + C::OFF_Q + lane * C::kBoxQ_B, &tmQ, lane * 64, w.hd * g, w.t.q_tok, bar(P_Q));
                ++q_act;
            }
            const int s = jg % C::KST;
            const uint32_t full = is_v ? v_full(s) : k_full(s);
            if (jg >= C::KST &&
                !(ok = wait_bar_warp(is_v ? v_empty(s) : k_empty(s), (jg / C::KST - 1) & 1, abort_flag, err)))
                break;
            const int tile = w.t.n_first + j;
            const uint32_t dst = ring + s * C::kTileKV_B;
            if (lane == 0)
                ptx::mbar_arrive_expect_tx(full, kPaged ? (uint32_t)(live * pr) * 128u * C::BOXES : C::kTileKV_B);
            __syncwarp();
            if constexpr (kPaged) {
                // keys before the window of the unit's first row may have lost their pages: they
                // are masked, and read as zeros (page `pages`) whatever the table says
                const int k_lo = a.window > 0 ? w.t.pos0 - a.window + 1 : 0;
                const int row8 = tiles_page > 1 ? tile % tiles_page * (BN / 8) : 0;
                bool bad = false;
#pragma unroll
                for (int i = 0; i < kPieces; ++i) {
                    const int c = lane + 32 * i, b = c / kPerPage;
                    if (b >= live) continue;
                    const int pg = tile * BN + (b + 1) * pr <= k_lo ? a.pages : page_checked(page[i], a.pages, &bad);
                    if constexpr (kGroup) {
                        tma_load_5d(dst + b * pr * (D * 2), map, w.hd * hs, 0, 0, row8, pg, full);
                    } else {
                        const int x = c % kPerPage;
                        tma_load_4d(dst + x * C::kBoxKV_B + b * pr * 128, map, x * 64, w.hd, row8 * 8, pg, full);
                    }
                }
                if (bad) atomicOr(err, kErrPage);
            } else if (lane < C::BOXES) {
                ptx::tma_load_3d(dst + lane * C::kBoxKV_B, map, lane * 64, w.hd, w.t.k_base + tile * BN, full);
            }
            ++jg;
            if (++j == w.j1) {
                do more = w.next();
                while (more && w.tiles() == 0);
                if (more) {
                    j = w.j0;
                    // the next item's Q tile to L2: the S products wait for its load
                    if (!is_v && lane < C::BOXES) tma_prefetch_3d(&tmQ, lane * 64, w.hd * g, w.t.q_tok);
                }
            }
            if (more) look_up();
        }
        __syncwarp();
        // never leave copies in flight into shared memory that is about to be released
        if (lane == 0) {
            if (q_act > 0) drain_wait(bar(P_Q), (q_act - 1) & 1);
            for (int k = jg - C::KST < 0 ? 0 : jg - C::KST; k < jg; ++k)
                drain_wait(is_v ? v_full(k % C::KST) : k_full(k % C::KST), (k / C::KST) & 1);
        }
        __syncwarp();
    } else if (warp == kWarpMma || warp == kWarpPv) {
        // ------------------------------------------------------------ MMA issuers
        // One warp issues S = Q K^T, another O += P V, so that each hides the other's waits.  S
        // of tile jg goes into buffer jg % NB once the P V product of tile jg - NB has read P
        // out of it; the P V product runs once the softmax has packed P.
        if (lane == 0 && !*abort_flag) {
            constexpr uint32_t ID_S = ptx::idesc_f16(BM, BN, kOpBF16, false, false);
            constexpr uint32_t ID_PV = ptx::idesc_f16(BM, D, kOpBF16, false, true);
            auto desc_add = [](uint64_t d, uint32_t bytes) { return d + (bytes >> 4); };
            bool ok = true;
            int jg = 0, ka = 0;
            FwdWalk w;
            bool more = w.init(share, blockIdx.x, a.H_kv, geo.overhead);
            if (warp == kWarpMma) {
                const uint64_t dQ_k = ptx::sw128_desc(sbase + C::OFF_Q, 16, 1024);
                const uint64_t dK_k = ptx::sw128_desc(sbase + C::OFF_K, 16, kRow8);
                [[maybe_unused]] int q_loads = 0;
                for (; ok && more; more = w.next()) {
                    const int nt = w.tiles();
                    if (nt == 0) continue;
                    if constexpr (kQ8) {  // no other warp loads Q
                        if (ka > 0 && !(ok = wait_bar(bar(P_QE), (ka - 1) & 1, abort_flag, err))) break;
                        ptx::mbar_arrive_expect_tx(bar(P_Q), (uint32_t)(geo.tpt * g) * 128u * C::BOXES);
#pragma unroll
                        for (int x = 0; x < C::BOXES; ++x)
                            ptx::tma_load_3d(sbase + C::OFF_Q + x * C::kBoxQ_B, &tmQ, x * 64, w.hd * g, w.t.q_tok, bar(P_Q));
                        q_loads = ka + 1;
                    }
                    if (!(ok = wait_bar(kConvQ ? q_conv : bar(P_Q), ka & 1, abort_flag, err))) break;
                    for (int j = 0; j < nt; ++j, ++jg) {
                        const int s = jg % C::KST;
                        if (!(ok = wait_bar(k_full(s), (jg / C::KST) & 1, abort_flag, err))) break;
                        if (jg >= NB && !(ok = wait_bar(bar(P_PV0 + jg % NB), (jg / NB - 1) & 1, abort_flag, err)))
                            break;
                        ptx::tc_fence_after();
                        const uint32_t so = (uint32_t)s * C::kTileKV_B;
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t kq = (kk / 4) * C::kBoxQ_B + (kk % 4) * 32;
                            const uint32_t kv = (kk / 4) * kBlk + (kk % 4) * 32;
                            ptx::mma_ss(tmem + C::TM_S + (jg % NB) * 128, desc_add(dQ_k, kq), desc_add(dK_k, so + kv),
                                        ID_S, kk > 0);
                        }
                        ptx::mma_commit(bar(P_S0 + jg % NB));
                        ptx::mma_commit(k_empty(s));
                    }
                    if (!ok) break;
                    ptx::mma_commit(bar(P_QE));
                    ++ka;
                }
                // every S product is read by a P V product, so all are complete once the other
                // issuer has drained
                if (kQ8 && q_loads > 0) drain_wait(bar(P_Q), (q_loads - 1) & 1);
            } else {
                const uint64_t dV_mn = ptx::sw128_desc(sbase + C::OFF_V, kBlk, kRow8);
                for (; ok && more; more = w.next()) {
                    const int nt = w.tiles();
                    if (nt == 0) continue;
                    for (int j = 0; j < nt; ++j, ++jg) {
                        const int s = jg % C::VST;
                        if (!(ok = wait_bar(v_full(s), (jg / C::VST) & 1, abort_flag, err))) break;
                        if (!(ok = wait_bar(bar(P_P0 + jg % NB), (jg / NB) & 1, abort_flag, err))) break;
                        // the first product of an item overwrites O: the epilogue of the
                        // previous item must have read it
                        if (j == 0 && ka > 0 && !(ok = wait_bar(bar(P_OFREE), (ka - 1) & 1, abort_flag, err))) break;
                        ptx::tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < BN / 16; ++kk)
                            ptx::mma_ts(tmem + C::TM_O, tmem + C::TM_S + (jg % NB) * 128 + packed_col<BN>(kk),
                                        desc_add(dV_mn, (uint32_t)s * C::kTileKV_B + kk * 2 * kRow8), ID_PV,
                                        (j > 0 || kk > 0) ? 1u : 0u);
                        ptx::mma_commit(bar(P_PV0 + jg % NB));
                        ptx::mma_commit(v_empty(s));
                    }
                    if (!ok) break;
                    ptx::mma_commit(bar(P_OFULL));
                    ++ka;
                }
                ptx::mma_commit(bar(P_FINAL));  // no MMA may still write TMEM when it is released
                drain_wait(bar(P_FINAL), 0);
            }
        }
        __syncwarp();
    }
    } else if (warp < kWarpEpi) {
        // ------------------------------------------------------------ softmax
        // Two threads per row, in warps w and w + 4 (of one TMEM lane quadrant), each half of a
        // tile's key columns.  (One thread per row took 1620 cycles a tile, mostly latency that
        // one warp per scheduler cannot hide; the two products of a tile take 1310.)
        //
        // The two need one reference m for their exponentials.  It need not be the max: exp2(x -
        // m) keeps its relative precision and only must not overflow.  So m is the max over the
        // first tile in which the row sees a key, and is found anew only when a row's half sum
        // over a tile exceeds kMaxSum (which bounds every P, also for fp16); in between the two
        // threads agree that it did not with one barrier.  S stays in TMEM until P replaces it.
        // A timeout never leaves the loop, so that the partner is not left at a barrier: all
        // waits return at once then.
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_SOFT));
        constexpr int HN = BN / 2;  // columns of a thread
        const int hf = warp >> 2, qd = warp & 3;
        const int t = qd * 32 + lane;  // TMEM lane == row of the tile
        const uint32_t lane_off = (uint32_t)(qd * 32) << 16;
        const uint32_t pair = kPairBarrier + qd;
        const int ti = t / g;  // token of the row
        const float scale_log2 = a.scale * 1.4426950408889634f;
        float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ROW);
        volatile float* xch = reinterpret_cast<volatile float*>(smem + C::OFF_XCH) + t;
        int jg = 0, ka = 0;
        FwdWalk w;
        bool more = !(sbase & 1023u) && w.init(share, blockIdx.x, a.H_kv, geo.overhead);
        for (; more; more = w.next()) {
            const bool row_valid = t < w.t.n_tok * g;
            const bool warp_live = qd * 32 < w.t.n_tok * g;
            const int nt = w.tiles();
            if (nt == 0) continue;
            // position of the request's first new token, and the masks of the row's token
            [[maybe_unused]] int ctx = 0;
            [[maybe_unused]] const unsigned long long* sees = nullptr;
            if constexpr (kTree) {
                ctx = w.t.pos0 - (w.t.q_tok - a.cu_q[w.t.n]);
                sees = a.tree + (size_t)(w.t.q_tok + (row_valid ? ti : 0)) * a.tree_words;
            }
            [[maybe_unused]] float scale_row = scale_log2;
            float m_run = -INFINITY;  // reference of the row's exponentials, in units of s * log2(e)
            float l_run = 0.f;        // sum of exp2(x - m_run) over this thread's columns
            for (int j = 0; j < nt; ++j, ++jg) {
                const uint32_t buf = tmem + C::TM_S + (jg % NB) * 128 + lane_off + hf * HN;
                const int n0 = (w.t.n_first + w.j0 + j) * BN;
                const int k_live = w.t.S_k - n0;  // keys of the sequence from this tile on
                int c_lo, c_hi;
                visible_keys(w.t.pos0 + ti - n0, a.causal, a.window, c_lo, c_hi);
                c_lo = max(c_lo, 0) - hf * HN;
                c_hi = min(c_hi, k_live) - hf * HN;
                const unsigned c_span = c_hi > c_lo ? (unsigned)(c_hi - c_lo) : 0u;
                const bool masked = __any_sync(0xffffffffu, !(c_lo <= 0 && c_hi >= HN));
                // a tile with new tokens: the thread's columns that the row's token sees, a bit each
                [[maybe_unused]] unsigned long long see = 0ull;
                [[maybe_unused]] const bool treed = kTree && n0 + BN > ctx;
                if constexpr (kTree)
                    if (treed) see = tree_columns<HN>(sees, a.tree_words, n0 + hf * HN - ctx);
                wait_bar_warp(bar(P_S0 + jg % NB), (jg / NB) & 1, abort_flag, err);
                [[maybe_unused]] float scale_tile = 0.f, v_exp = 0.f, v_unit = 1.f;
                [[maybe_unused]] bool far = false;
                if constexpr (kQ8) {
                    // what Q's row was multiplied by is taken out of the scores again
                    if (kConvQ && j == 0)
                        scale_row = scale_log2 * reinterpret_cast<volatile const float*>(smem + C::OFF_QS)[(ka & 3) * BM + t];
                    // K = K' 2^ek, V = V' 2^ev of the tile's operands K', V': the scores take 2^ek, and the
                    // exponentials, which stand for P 2^ev, ev
                    const uint32_t top = *reinterpret_cast<volatile const uint32_t*>(smem + C::OFF_TOP + (jg & 7) * 4);
                    // never 0, which would make NaN of the -inf of masked scores: not for a tile whose keys are
                    // all zeros (ek is 0 - 127 then, and no float's), nor where the product falls below the
                    // normal numbers (every score rounds to 0 either way)
                    scale_tile = fmaxf(scale_row * __uint_as_float((top & 0xffu) << 23), 1.17549435e-38f);
                    v_exp = (float)((int)(top >> 8 & 0xffu) - 127);
                    v_unit = __uint_as_float((254u - (top >> 8 & 0xffu)) << 23);  // 2^-ev
                    far = (top & kTopFar) != 0;
                }
                if (!kQ8 && k_live < BN) {
                    // V rows behind the last key: zeros, once the loads have landed
                    const int s = jg % C::VST;
                    wait_bar_warp(v_full(s), (jg / C::VST) & 1, abort_flag, err);
                    if (hf == 0 && t < BN && t >= k_live) {
#pragma unroll
                        for (int x = 0; x < C::BOXES; ++x)
#pragma unroll
                            for (int q = 0; q < 8; ++q)
                                *reinterpret_cast<uint4*>(smem + C::OFF_V + s * C::kTileKV_B + x * kBlk +
                                                          (t >> 3) * kRow8 + (t & 7) * 128 + q * 16) =
                                    make_uint4(0u, 0u, 0u, 0u);
                    }
                    ptx::fence_proxy_async_smem();
                }
                ptx::tc_fence_after();
                if (warp_live) {
                    float alpha = 1.f, sum = 0.f;
                    bool rescale = false;
                    uint32_t Pp[HN / 2];
                    auto load = [&](uint32_t* r) {
#pragma unroll
                        for (int c = 0; c < HN / 32; ++c) ptx::tmem_ld32p(buf + c * 32, r + c * 32);
                        ptx::tmem_wait_ld();
                        if (masked) {
#pragma unroll
                            for (int c = 0; c < HN; ++c)
                                r[c] = (unsigned)(c - c_lo) < c_span ? r[c] : __float_as_uint(-INFINITY);
                        }
                        if constexpr (kTree) {
                            if (treed) {
#pragma unroll
                                for (int c = 0; c < HN; ++c)
                                    r[c] = (see >> c & 1ull) ? r[c] : __float_as_uint(-INFINITY);
                            }
                        }
                    };
                    auto exps = [&](const uint32_t* r) {
                        const float m_use = m_run == -INFINITY ? 0.f : m_run;
                        const float sc = kQ8 ? scale_tile : scale_log2, nm = kQ8 ? v_exp - m_use : -m_use;
                        const float2 sc2 = make_float2(sc, sc);
                        const float2 nm2 = make_float2(nm, nm);
                        float2 sum2[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                                          make_float2(0.f, 0.f)};
#pragma unroll
                        for (int c = 0; c < HN; c += 2) {
                            const float2 x =
                                __ffma2_rn(make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), sc2, nm2);
                            const float2 pp = make_float2(ptx::ex2(x.x), ptx::ex2(x.y));
                            sum2[(c >> 1) & 3] = __fadd2_rn(sum2[(c >> 1) & 3], pp);
                            Pp[c / 2] = pack2<kOpBF16>(pp.x, pp.y);
                        }
                        const float2 s2 = __fadd2_rn(__fadd2_rn(sum2[0], sum2[1]), __fadd2_rn(sum2[2], sum2[3]));
                        sum = s2.x + s2.y;
                    };
                    // the max of both halves, by way of the second half's thread
                    auto both_halves = [&](float mx) {
                        if (hf == 1) *xch = mx;
                        __syncwarp();
                        ptx::named_bar_sync(pair, 64);
                        if (hf == 0) *xch = mx = fmaxf(mx, *xch);
                        __syncwarp();
                        ptx::named_bar_sync(pair, 64);
                        if (hf == 1) mx = *xch;
                        return mx;
                    };
                    auto refer_to = [&](float mx) {
                        rescale = mx > m_run;
                        if (rescale) {
                            alpha = m_run == -INFINITY ? 0.f : ptx::ex2(m_run - mx);
                            m_run = mx;
                        }
                    };
                    if (kQ8 && far) {
                        const uint16_t* own = reinterpret_cast<const uint16_t*>(smem + C::OFF_FAR) + (jg & 7) * BN + hf * HN;
                        refer_to(both_halves(far_scores<HN>(buf, own, scale_row, [&](int c) {
                                     return (unsigned)(c - c_lo) < c_span && (!treed || (see >> c & 1ull));
                                 })) - kQ8Lift);
                        l_run = l_run * alpha + far_weights<HN, kOpBF16>(buf, own, m_run == -INFINITY ? 0.f : m_run);
                    } else {
                        bool done = false;
                        // both threads of a row have the same m, so both warps decide alike
                        if (j > 0 && !__any_sync(0xffffffffu, row_valid && m_run == -INFINITY)) {
                            uint32_t r[HN];
                            load(r);
                            exps(r);
                            __syncwarp();
                            done = ptx::named_bar_and(pair, 64, !(row_valid && sum > (kQ8 ? kQ8MaxSum : kMaxSum)));
                        }
                        if (!done) {
                            uint32_t r[HN];
                            load(r);
                            float mx8[8];
#pragma unroll
                            for (int q = 0; q < 8; ++q) mx8[q] = -INFINITY;
#pragma unroll
                            for (int c = 0; c < HN; c += 2)
                                mx8[(c >> 1) & 7] = fmax3(mx8[(c >> 1) & 7], __uint_as_float(r[c]), __uint_as_float(r[c + 1]));
                            float mx = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                                             fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7])));
                            mx = both_halves(mx);
                            refer_to(mx == -INFINITY ? -INFINITY : kQ8 ? fmaf(mx, scale_tile, v_exp - kQ8Lift) : mx * scale_log2);
                            exps(r);
                        }
                        l_run = l_run * alpha + (kQ8 ? sum * v_unit : sum);
#pragma unroll
                        for (int c = 0; c < HN / 2; c += 16) ptx::tmem_st16(buf + c, *reinterpret_cast<uint32_t(*)[16]>(Pp + c));
                    }
                    // rescale the O row before the next P V product accumulates into it (each
                    // thread half of the columns)
                    if (j > 0 && __any_sync(0xffffffffu, rescale)) {
                        wait_bar_warp(bar(P_PV0 + (jg - 1) % NB), ((jg - 1) / NB) & 1, abort_flag, err);
                        ptx::tc_fence_after();
#pragma unroll
                        for (int c = 0; c < D / 64; ++c) {
                            uint32_t o[32];
                            const uint32_t at = tmem + C::TM_O + lane_off + hf * (D / 2) + c * 32;
                            ptx::tmem_ld32p(at, o);
                            ptx::tmem_wait_ld();
#pragma unroll
                            for (int kk = 0; kk < 32; ++kk) o[kk] = __float_as_uint(__uint_as_float(o[kk]) * alpha);
                            ptx::tmem_st32(at, o);
                        }
                    }
                    ptx::tmem_wait_st();
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(P_P0 + jg % NB));
            }
            // (m, l) of the row to the epilogue, once the slot's values of two items ago have been
            // read (items of a tile or two can be through here before the epilogue of the first
            // of them has begun)
            if (hf == 1) *xch = l_run;
            __syncwarp();
            ptx::named_bar_sync(pair, 64);
            if (hf == 0) {
                if (ka > 1) wait_bar_warp(bar(P_MR0 + (ka & 1)), ((ka >> 1) - 1) & 1, abort_flag, err);
                ml[(ka & 1) * BM + t] = make_float2(m_run, l_run + *xch);
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(P_ML0 + (ka & 1)));
            }
            __syncwarp();
            ptx::named_bar_sync(pair, 64);  // the exchange word is free again
            ++ka;
        }
    } else {
        // ------------------------------------------------------------ epilogue
        // O = acc / l and LSE = (m + log2 l) ln 2 of a whole item; of a cut one the raw
        // accumulator with (m, l), and the last part to arrive joins them.  Meanwhile the
        // softmax warps are at the next item; its first P V product waits for O to be read.
        if constexpr (C::REGS_EPI > C::REGS)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_EPI));
        else
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_EPI));
        const int t = threadIdx.x - kWarpEpi * 32;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const int ti = t / g, th = t - ti * g;  // token and head of the row
        const bool wide = ((reinterpret_cast<uintptr_t>(a.O) | (a.o.tok * 2) | (a.o.head * 2)) & 31) == 0;
        float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ROW);
        int ka = 0;
        FwdWalk w;
        bool more = !*abort_flag && w.init(share, blockIdx.x, a.H_kv, geo.overhead);
        for (; more; more = w.next()) {
            const int rows = w.t.n_tok * g;
            const bool row_valid = t < rows;
            const bool warp_live = (warp & 3) * 32 < rows;
            const bool has = w.tiles() > 0;
            const bool whole = w.whole();
            float m_run = -INFINITY, l_run = 0.f;
            if (has) {
                // all four warps take the same decision (they meet at a barrier below)
                bool ok = wait_bar_warp(bar(P_ML0 + (ka & 1)), (ka >> 1) & 1, abort_flag, err);
                ok = ok && wait_bar_warp(bar(P_OFULL), ka & 1, abort_flag, err);
                __syncwarp();
                if (!ptx::named_bar_and(kEpiBarrier, 128, ok)) break;
                const float2 x = ml[(ka & 1) * BM + t];
                m_run = x.x, l_run = x.y;
                __syncwarp();
                // (of a whole item; a cut one's slot serves as scratch below)
                if (whole && lane == 0) ptx::mbar_arrive(bar(P_MR0 + (ka & 1)));
                ++ka;
            }
            ptx::tc_fence_after();
            const float inv_l = inv_sum(l_run);
            const int tok = w.t.q_tok + ti, head = w.hd * g + th;
            const int slot = 2 * (int)blockIdx.x + (w.j0 == 0 ? 1 : 0);
            if (warp_live) {
                T* Orow = static_cast<T*>(a.O) + (long long)tok * a.o.tok + (long long)head * a.o.head;
                float* Prow = plan.part_o + ((size_t)slot * BM + t) * D;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    if (has) {
                        ptx::tmem_ld32p(tmem + C::TM_O + lane_off + c * 32, o);
                        ptx::tmem_wait_ld();
                        if (c == D / 32 - 1) {  // O read: the next item may overwrite it
                            ptx::tc_fence_before();
                            __syncwarp();
                            if (lane == 0) ptx::mbar_arrive(bar(P_OFREE));
                        }
                    } else {
#pragma unroll
                        for (int kk = 0; kk < 32; ++kk) o[kk] = 0u;
                    }
                    if (row_valid && whole) {
                        if (c * 32 < a.d) {
                            uint32_t w[16];
#pragma unroll
                            for (int kk = 0; kk < 16; ++kk)
                                w[kk] = pack2<kBF16>(__uint_as_float(o[2 * kk]) * inv_l,
                                                     __uint_as_float(o[2 * kk + 1]) * inv_l);
                            if (wide) {
                                st_global_v8(Orow + c * 32, w);
                                st_global_v8(Orow + c * 32 + 16, w + 8);
                            } else {
#pragma unroll
                                for (int u = 0; u < 4; ++u)
                                    *reinterpret_cast<uint4*>(Orow + c * 32 + u * 8) =
                                        make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]);
                            }
                        }
                    } else if (row_valid) {
#pragma unroll
                        for (int u = 0; u < 4; ++u) st_global_v8(Prow + c * 32 + u * 8, o + u * 8);
                    }
                    __syncwarp();
                }
                if (row_valid) {
                    if (whole)
                        a.LSE[(size_t)head * a.T_q + tok] = lse_of(m_run, l_run);
                    else
                        plan.part_ml[(size_t)slot * BM + t] = make_float2(part_max(m_run, l_run), l_run);
                    // without a key the accumulator is 0 times V, which an infinity in V makes NaN
                    if (whole && has && l_run == 0.f)
#pragma unroll 1
                        for (int c = 0; c < a.d; c += 8) *reinterpret_cast<uint4*>(Orow + c) = make_uint4(0u, 0u, 0u, 0u);
                }
            } else if (has && lane == 0) {
                ptx::mbar_arrive(bar(P_OFREE));
            }
            if (!whole) {
                int first, count;
                w.parts(first, count);
                __threadfence();
                __syncwarp();
                ptx::named_bar_sync(kEpiBarrier, 128);
                if (t == 0) *last_flag = arrive_part(&plan.done[first], plan.tag, count);
                __syncwarp();
                ptx::named_bar_sync(kEpiBarrier, 128);
                if (*last_flag) {
                    __threadfence();
                    join_parts<T, 128, BM, D, 4>(a, plan, w.t, w.hd * g, g, rows, first, count, t,
                                              ml + ((ka - 1) & 1) * BM, [] {
                                                  __syncwarp();
                                                  ptx::named_bar_sync(kEpiBarrier, 128);
                                              });
                    __syncwarp();
                    ptx::named_bar_sync(kEpiBarrier, 128);
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(P_MR0 + ((ka - 1) & 1)));
            }
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == kWarpMma) ptx::tmem_dealloc(tmem, kTmemCols);
}

// ---------------------------------------------------------------- host side
bool encode(CUtensorMap* m, const void* base, CUtensorMapDataType dt, int rank, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box) {
    TmaEncodeTiledFn enc = tma_encode_fn();
    const cuuint32_t one[5] = {1, 1, 1, 1, 1};
    return enc && enc(m, dt, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, one,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D, bool kPaged, bool kGroup, bool kTree, bool kQ8 = false>
cudaError_t launch_t(const PackedFwd& a, void* ws, size_t* bytes, cudaStream_t st) {
    using C = PCfg<D, kQ8>;
    constexpr uint32_t kSmem = C::OFF_BAR + (P_SLOT0 + 2 * C::KST + 2 * C::VST + (kQ8 ? 1 + 2 * C::INFO : 0)) * 8 + 16;
    static_assert(kSmem <= 232448, "shared memory budget");
    const int g = a.H / a.H_kv;
    FwdGeom geo;
    geo.rows = BM;
    geo.tpt = BM / g;
    geo.bn = C::BN;
    geo.heads = a.H_kv;
    geo.ctas = sm_count();
    geo.D = D;
    geo.min_chunk = 2;
    // filling the pipeline and the epilogue cost about three tiles' time.  With 2 (3 for items
    // of one tile) mixed prompts took 328 us against 333, chunks over a cache 119 against 115
    geo.overhead = 3;
    const long long units = plan_units(a, geo);
    geo.self = units <= kSelfUnits && a.N <= kSelfUnits;
    FwdPlan plan;
    *bytes = fwd_plan_layout(a, geo, ws, &plan);
    if (ws == nullptr) return cudaSuccess;
    plan.tag = next_tag();
    const CUtensorMapDataType dt =
        TypeTraits<T>::kId == FA_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    CUtensorMap tq, tk = {}, tv = {};
    bool ok;
    {
        const cuuint64_t dims[3] = {(cuuint64_t)a.d, (cuuint64_t)a.H, (cuuint64_t)a.T_q};
        const cuuint64_t str[2] = {(cuuint64_t)a.q.head * 2, (cuuint64_t)a.q.tok * 2};
        const cuuint32_t box[3] = {64, (cuuint32_t)g, (cuuint32_t)geo.tpt};
        ok = encode(&tq, a.Q, dt, 3, dims, str, box);
    }
    const struct {
        CUtensorMap* m;
        const void* p;
        RowStride s;
        long long page;
    } kv[2] = {{&tk, a.K, a.k, a.k_page}, {&tv, a.V, a.v, a.v_page}};
    for (int i = 0; i < 2 && !kQ8; ++i) {
        if constexpr (kGroup) {
            // columns of a head (its offset is part of the column coordinate), 8 rows, 64-column
            // blocks, groups of 8 rows, pages
            const cuuint64_t row = (cuuint64_t)kv[i].s.tok * 2;
            const cuuint64_t dims[5] = {(cuuint64_t)((a.H_kv - 1) * kv[i].s.head + 64), 8, D / 64,
                                        (cuuint64_t)(a.page_size / 8), (cuuint64_t)a.pages};
            const cuuint64_t str[4] = {row, 128, row * 8, (cuuint64_t)kv[i].page * 2};
            const cuuint32_t box[5] = {64, 8, D / 64, (cuuint32_t)((a.page_size < C::BN ? a.page_size : C::BN) / 8), 1};
            ok = ok && encode(kv[i].m, kv[i].p, dt, 5, dims, str, box);
        } else if constexpr (kPaged) {
            const cuuint64_t dims[4] = {(cuuint64_t)a.d, (cuuint64_t)a.H_kv, (cuuint64_t)a.page_size,
                                        (cuuint64_t)a.pages};
            const cuuint64_t str[3] = {(cuuint64_t)kv[i].s.head * 2, (cuuint64_t)kv[i].s.tok * 2,
                                       (cuuint64_t)kv[i].page * 2};
            const cuuint32_t box[4] = {64, 1, (cuuint32_t)(a.page_size < C::BN ? a.page_size : C::BN), 1};
            ok = ok && encode(kv[i].m, kv[i].p, dt, 4, dims, str, box);
        } else {
            const cuuint64_t dims[3] = {(cuuint64_t)a.d, (cuuint64_t)a.H_kv, (cuuint64_t)(a.T_k > 0 ? a.T_k : 1)};
            const cuuint64_t str[2] = {(cuuint64_t)kv[i].s.head * 2, (cuuint64_t)kv[i].s.tok * 2};
            const cuuint32_t box[3] = {64, 1, (cuuint32_t)C::BN};
            ok = ok && encode(kv[i].m, a.T_k > 0 ? kv[i].p : a.Q, dt, 3, dims, str, box);
        }
    }
    if (!ok) return cudaErrorInvalidValue;
    cudaError_t e;
    if (!geo.self && (e = launch_fwd_plan(a, geo, plan, st)) != cudaSuccess) return e;
    auto kern = packed_fwd_kernel<T, D, kPaged, kGroup, kTree, kQ8>;
    static std::atomic<uint64_t> ready{0};
    if ((e = allow_smem(kern, (int)kSmem, ready)) != cudaSuccess) return e;
    // programmatic dependent launch: barriers and TMEM are set up while the kernel before runs
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)geo.ctas);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, tq, tk, tv, a, plan, geo, (int)units);
}

// The paged instances (kTree: those with masks).
template <typename T, bool kTree>
cudaError_t launch_paged(const PackedFwd& a, void* ws, size_t* bytes, cudaStream_t st) {
    const int D = a.d == 256 ? 256 : tc_head_dim(a.d);
    // head dims 32 and 96 keep a box per 64 columns, whose missing columns read as zeros
    const bool group = a.d == D && (long long)a.H_kv * (a.k.head > a.v.head ? a.k.head : a.v.head) < (1ll << 31);
    if (D == 64) return launch_t<T, 64, true, false, kTree>(a, ws, bytes, st);
    if (D == 128 && group) return launch_t<T, 128, true, true, kTree>(a, ws, bytes, st);
    if (D == 128) return launch_t<T, 128, true, false, kTree>(a, ws, bytes, st);
    if (D == 256 && group) return launch_t<T, 256, true, true, kTree>(a, ws, bytes, st);
    if (D == 256) return launch_t<T, 256, true, false, kTree>(a, ws, bytes, st);
    return cudaErrorInvalidValue;
}

}  // namespace
}  // namespace fa
