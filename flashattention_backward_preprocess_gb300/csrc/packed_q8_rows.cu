// packed_q8_rows.cu -- attention over an 8-bit cache for steps of few rows (a token or a few for each
// request): packed_fwd_tc.cuh's plan, items and joins, but each warp copies, converts and multiplies its
// own keys, with no operand in shared memory and no warp waiting for another.
//
// An item's rows (up to 16: tpt tokens x the g heads of a key/value head) are one 16-row operand of
// mma.sync m16n8k16, whose fragments a thread can load for itself.  (tcgen05 reads 128 rows of which
// such a step fills g, and takes its operands from shared memory: the 8-bit rows would have to be
// written there as fp16 first.)  Warp w of a CTA's W takes keys [16 w, 16 w + 16) of each tile of 16 W, with
// a max, a sum and an accumulator of its own; they meet once, at the item's end.
//   * K: the products of Q K^T run over d in an order in which a lane's operands are 16 bytes next to
//     each other: lane (q = lane / 4, t = lane % 4) takes bytes [64 x + 16 t, + 16) of keys q and q + 8.
//   * V: the output columns are numbered so that a lane needs bytes [q D / 8, + D / 8) of its four keys
//     2t, 2t + 1, 2t + 8, 2t + 9: whole 128-byte lines again; two bytes of two keys are paired by a
//     byte permutation, and pairs made fp16 by one conversion.
//   * exponents: e_k goes into the score of its key.  With y = score + e_v the weight P' = 2^(y - m)
//     stands for P 2^e_v and multiplies V's numbers as they are; the row sum takes P' 2^-e_v.  m is
//     the max of y less 8, looked at anew when a y exceeds m by 15: P' <= 2^15 fits fp16, whose fixed
//     step below 2^-14 is 2^-33 of the row's largest weight.
//   * Q is fp16, a bf16 row times a power of two (packed_q8.cuh says why).
// Bytes come through a ring in shared memory, kStages tiles of a warp's 4 KB, by asynchronous copies;
// every thread copies the numbers that it will read itself, so no warp waits for another.  Twelve warps a
// SM: in three CTAs of four (tiles of 64 keys) when there are many items, whose ends then overlap; in one of
// twelve (192 keys) when there are few, since an item is cut into as many parts as CTAs share it, and
// whoever joins the parts reads them all.
//
// Bound by latency at three warps a scheduler (520 instructions per warp and 16 keys, 0.43 issued a cycle and
// scheduler; of 6.7 cycles between two of a warp 2.0 are fixed latencies, 1.5 memory's), then DRAM.  Measured
// in a replayed graph, bf16, H = 32, H_kv = 8, d = 128: 64 requests, one token each, over 0.57 GB of cache 141
// us (4.1 TB/s); one token of f16, H = 16, H_kv = 2, over 131072 keys 61 us; over 1024 keys 20 us.
#include <cuda_fp16.h>
#include <math.h>

#include "packed.cuh"
#include "packed_q8.cuh"

namespace fa {
namespace {

constexpr int RT = 16;  // rows of a tile; its keys: 16 per warp
// Warps of a CTA, CTAs per SM and stages of the ring: many items, few items
constexpr int kManyWarps = 4, kManyCtas = 3, kManyStages = 3;
constexpr int kFewWarps = 12, kFewCtas = 1, kFewStages = 4;
constexpr float kLift = 8.f, kRoom = 15.f;

// The first `live` of 16 bytes, zeros behind them.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(live ? 8u : 0u) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
__device__ __forceinline__ float quad_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x + __shfl_xor_sync(0xffffffffu, x, 2);
}
// Byte n of a word as an exponent: 2^(b - 127), 2^(127 - b).
__device__ __forceinline__ float up2(uint32_t w, int n) { return __uint_as_float((w >> (8 * n) & 0xffu) << 23); }
// b - 127 (2^23 + b as a float, less 2^23 + 127)
__device__ __forceinline__ float minus127(uint32_t w, int n) {
    return __uint_as_float(0x4b000000u | (w >> (8 * n) & 0xffu)) - 8388735.f;
}
__device__ __forceinline__ float down2(uint32_t w, int n) { return __uint_as_float((254u - (w >> (8 * n) & 0xffu)) << 23); }

// Joins the parts of a cut item (join_parts with few rows and many parts: one long request is cut over
// the whole grid).  Of kWarps warps each takes every kWarps-th part, 16 loads of a thread in flight, and
// they meet in s_o; joining one after another, 76 parts took 100 us.
template <typename T, int D, int kWarps>
__device__ __forceinline__ void join_rows(const PackedFwd& a, const FwdPlan& p, const FwdTile& tile, int head0, int g, int rows,
                                          int first, int count, float (*s_o)[RT][D + 4], float2* s_row) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    auto slot = [&](int k) { return (size_t)(k == 0 ? 2 * first + 1 : 2 * (first + k)) * RT; };
    {  // max and sum of a row: eight lanes each, every eighth part
        const int r = tid >> 3;
        float M = -INFINITY, L = 0.f;
        if (r < rows)
#pragma unroll 4
            for (int k = tid & 7; k < count; k += 8) {
                const float2 ml = __ldcg(&p.part_ml[slot(k) + r]);
                const float top = fmaxf(M, ml.x), base = top == -INFINITY ? 0.f : top;
                L = L * ptx::ex2(M - base) + ml.y * ptx::ex2(ml.x - base);  // a NaN max reaches the sum
                M = top;
            }
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) {
            const float M2 = __shfl_xor_sync(0xffffffffu, M, o), L2 = __shfl_xor_sync(0xffffffffu, L, o);
            const float top = fmaxf(M, M2), base = top == -INFINITY ? 0.f : top;
            // the same order in both lanes
            const bool low = (tid & o) == 0;
            const float la = (low ? L : L2) * ptx::ex2((low ? M : M2) - base), lb = (low ? L2 : L) * ptx::ex2((low ? M2 : M) - base);
            L = la + lb;
            M = top;
        }
        if ((tid & 7) == 0 && r < RT) {
            s_row[r] = make_float2(M == -INFINITY ? 0.f : M, inv_sum(L));
            if (r < rows) a.LSE[(size_t)(head0 + r % g) * a.T_q + tile.q_tok + r / g] = lse_of(M, L);
        }
    }
    __syncthreads();
    const int n4 = rows * (D / 4);
    for (int e0 = lane; e0 < n4; e0 += 128) {
        float4 s[4];
#pragma unroll
        for (int b = 0; b < 4; ++b) s[b] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = warp; k0 < count; k0 += 4 * kWarps) {
            float4 o[4][4];
            float f[4][4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const int k = k0 + u * kWarps, e = e0 + b * 32, r = e / (D / 4);
                    o[u][b] = make_float4(0.f, 0.f, 0.f, 0.f);
                    f[u][b] = 0.f;
                    if (k < count && e < n4) {
                        o[u][b] = __ldcg(reinterpret_cast<const float4*>(p.part_o + (slot(k) + r) * D) + e % (D / 4));
                        f[u][b] = __ldcg(&p.part_ml[slot(k) + r]).x;
                    }
                }
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const int k = k0 + u * kWarps, e = e0 + b * 32;
                    if (k >= count || e >= n4 || f[u][b] == -INFINITY) continue;
                    const float w = ptx::ex2(f[u][b] - s_row[e / (D / 4)].x);
                    s[b].x = fmaf(o[u][b].x, w, s[b].x), s[b].y = fmaf(o[u][b].y, w, s[b].y);
                    s[b].z = fmaf(o[u][b].z, w, s[b].z), s[b].w = fmaf(o[u][b].w, w, s[b].w);
                }
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int e = e0 + b * 32;
            if (e < n4) *reinterpret_cast<float4*>(&s_o[warp][e / (D / 4)][e % (D / 4) * 4]) = s[b];
        }
    }
    __syncthreads();
    for (int e = tid; e < n4; e += kWarps * 32) {
        const int r = e / (D / 4), c = e % (D / 4) * 4;
        if (c >= a.d) continue;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int v = 0; v < kWarps; ++v) {
            const float4 x = *reinterpret_cast<const float4*>(&s_o[v][r][c]);
            s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
        }
        const float inv = s_row[r].y;
        alignas(8) T out[4] = {TypeTraits<T>::from_f32(s.x * inv), TypeTraits<T>::from_f32(s.y * inv),
                               TypeTraits<T>::from_f32(s.z * inv), TypeTraits<T>::from_f32(s.w * inv)};
        *reinterpret_cast<uint2*>(static_cast<T*>(a.O) + (long long)(tile.q_tok + r / g) * a.o.tok +
                                  (long long)(head0 + r % g) * a.o.head + c) = *reinterpret_cast<const uint2*>(out);
    }
    __syncthreads();  // s_o is free again
}

// A warp's stage: K pieces [block][key half][lane], V pieces [key][lane], exponents of 16 keys of K, of V.
template <int D>
constexpr int kStageB = (D / 64) * 2 * 512 + 4 * 32 * (D / 8) + 32;
// Dynamic shared memory: the ring, where the accumulators meet and the plan is made as well.
template <int D, int kWarps, int kStages>
constexpr int kSmemB = kWarps * kStages * kStageB<D> > kWarps * RT * (D + 4) * 4 ? kWarps * kStages * kStageB<D>
                                                                               : kWarps * RT * (D + 4) * 4;

template <typename T, int D, bool kTree, int kWarps, int kCtas, int kStages>
__global__ void __launch_bounds__(kWarps * 32, kCtas)
    q8_rows_kernel(const PackedFwd a, const FwdPlan plan, const FwdGeom geo, int max_units) {
    constexpr int kThreads = kWarps * 32, KT = 16 * kWarps;
    constexpr int X = D / 64;   // 64-column blocks of a row
    constexpr int CH = D / 8;   // V's bytes of a key per lane, output tiles of 8 columns
    constexpr int LD = D + 4;
    constexpr int kB = kStageB<D>, kVOff = X * 2 * 512, kEOff = kVOff + 4 * 32 * CH;
    constexpr bool kScaleQ = TypeTraits<T>::kId == FA_BF16;
    extern __shared__ __align__(16) uint8_t smem[];
    float(*s_o)[RT][LD] = reinterpret_cast<float(*)[RT][LD]>(smem);
    __shared__ uint4 s_q[X * 4][32];  // operands of Q by product step and lane
    __shared__ float2 s_ml[kWarps][RT];
    __shared__ float2 s_row[RT];
    __shared__ int s_last;
    static_assert((int)sizeof(SelfPlan) <= kSmemB<D, kWarps, kStages>, "the plan is made there");
    static_assert(kB % 16 == 0, "16-byte copies");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, q = lane >> 2, t = lane & 3;
    const int g = a.H / a.H_kv;
    ptx::griddep_wait();
    FwdShare share;
    if (geo.self) {
        SelfPlan* sp = reinterpret_cast<SelfPlan*>(smem);
        plan_self<kThreads>(a, geo, plan, max_units, sp);
        share = sp->share;
        __syncthreads();
        if (a.fill) fill_rows<T>(a, share.W == 0, blockIdx.x * kThreads + tid, (long long)gridDim.x * kThreads);
    } else {
        share.read(plan, blockIdx.x);
    }
    const int shift = (a.page_size & (a.page_size - 1)) == 0 ? 31 - __clz(a.page_size) : -1;
    const uint8_t* Kb = static_cast<const uint8_t*>(a.K);
    const uint8_t* Vb = static_cast<const uint8_t*>(a.V);
    const uint32_t ring = ptx::smem_u32(smem) + warp * (kStages * kB);
    const uint8_t* ring_p = smem + warp * (kStages * kB);
    FwdWalk w;
    for (bool more = w.init(share, blockIdx.x, a.H_kv, geo.overhead); more; more = w.next()) {
        const int rows = w.t.n_tok * g, head0 = w.hd * g;
        // ---- Q: rows q and q + 8, 16 columns of each block, as fp16 operands
        float rs[2];  // of a row: scores to log2 units
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = q + 8 * h;
            const T* Qr = static_cast<const T*>(a.Q) + (long long)(w.t.q_tok + r / g) * a.q.tok + (long long)(head0 + r % g) * a.q.head;
            uint4 raw[X][2];
            float most = 0.f;
#pragma unroll
            for (int x = 0; x < X; ++x) {
                const int c = x * 64 + t * 16;
                const bool in = r < rows && c < a.d;
                raw[x][0] = in ? reinterpret_cast<const uint4*>(Qr + c)[0] : make_uint4(0u, 0u, 0u, 0u);
                raw[x][1] = in ? reinterpret_cast<const uint4*>(Qr + c)[1] : make_uint4(0u, 0u, 0u, 0u);
            }
            int n = 0;
            if (kScaleQ) {
#pragma unroll
                for (int x = 0; x < X; ++x)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t v = (&raw[x][i >> 2].x)[i & 3];
                        const float lo = fabsf(__uint_as_float(v << 16)), hi = fabsf(__uint_as_float(v & 0xffff0000u));
                        most = fmaxf(most, fmaxf(lo <= 3.4e38f ? lo : 0.f, hi <= 3.4e38f ? hi : 0.f));
                    }
                most = quad_max(most);
                n = most > 0.f ? min(100, 14 - ((__float_as_int(most) >> 23) - 127)) : 0;
            }
            const float s = __int_as_float((n + 127) << 23);
            rs[h] = a.scale * 1.4426950408889634f * __int_as_float((127 - n) << 23);
#pragma unroll
            for (int x = 0; x < X; ++x)
#pragma unroll
                for (int i = 0; i < 8; ++i) {  // columns 2i, 2i + 1 of the lane's 16
                    uint32_t v = (&raw[x][i >> 2].x)[i & 3];
                    if (kScaleQ) v = pack_half2(__uint_as_float(v << 16) * s, __uint_as_float(v & 0xffff0000u) * s);
                    if (warp == (i >> 1)) (&s_q[x * 4 + (i >> 1)][lane].x)[(i & 1) * 2 + h] = v;
                }
        }
        __syncthreads();
        uint4 qr[X * 4];
#pragma unroll
        for (int i = 0; i < X * 4; ++i) qr[i] = s_q[i][lane];
        const int ctx = kTree ? w.t.pos0 - (w.t.q_tok - a.cu_q[w.t.n]) : 0;
        const int k_lo = a.window > 0 ? w.t.pos0 - a.window + 1 : 0;  // no row sees an earlier key
        const int* table = a.table + (size_t)w.t.n * a.max_pages;
        const int nt = w.tiles();
        const int first = (w.t.n_first + w.j0) * KT + warp * 16;  // this warp's first key
        // ---- loads.  A warp's 16 keys of a tile lie on one page (page_size % 16 == 0).
        auto entry_of = [&](int j) {  // table entry of the warp's keys in tile j; -2: no key there that a row sees
            const int key0 = first + j * KT;
            if (j >= nt || key0 >= w.t.S_k || key0 + 16 <= k_lo) return -2;
            const int e = shift >= 0 ? key0 >> shift : key0 / a.page_size;
            return e < a.max_pages ? table[e] : -1;
        };
        // keys that all rows see: [all_lo, all_hi)
        const int all_lo = a.window > 0 ? w.t.pos0 + w.t.n_tok - a.window : 0;
        const int all_hi = min(min(w.t.S_k, kTree ? ctx : kOpen),
                               a.causal ? w.t.pos0 + 1 : a.window > 0 ? w.t.pos0 + a.window : kOpen);
        auto page_at = [&](int entry) -> int {  // the page; `pages`: zeros; -1: no key
            if (entry == -2) return -1;
            bool bad = false;
            const int pg = page_checked(entry, a.pages, &bad);
            if (bad && lane == 0) atomicOr(a.err, kErrPage);
            return pg;
        };
        // the warp's keys of tile j, on page pg, into stage `st`
        const uint8_t* Kl = Kb + (long long)w.hd * a.k.head + q * a.k.tok + t * 16;
        const uint8_t* Vl = Vb + (long long)w.hd * a.v.head + 2 * t * a.v.tok + q * CH;
        auto fetch = [&](int j, int pg, int st) {
            const int key0 = first + j * KT, in0 = shift >= 0 ? key0 & (a.page_size - 1) : key0 % a.page_size;
            const int left = pg < a.pages ? w.t.S_k - key0 : 0;  // keys from here on
            const uint32_t dst = ring + st * kB;
            const uint8_t* pk = Kl + pg * a.k_page + in0 * a.k.tok;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int x = 0; x < X; ++x) {
                    const bool in = q + 8 * i < left && x * 64 + t * 16 < a.d;
                    cp_async16(dst + (x * 2 + i) * 512 + lane * 16, in ? pk + x * 64 : Kb, in ? 16u : 0u);
                }
                pk += 8 * a.k.tok;
            }
            const uint8_t* pv = Vl + pg * a.v_page + in0 * a.v.tok;
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                const int r = 2 * t + (n & 1) + (n >> 1) * 8;
                const bool in = r < left && q * CH < a.d;
                const uint32_t to = dst + kVOff + (n * 32 + lane) * CH;
                if constexpr (CH == 16)
                    cp_async16(to, in ? pv : Vb, in ? 16u : 0u);
                else
                    cp_async8(to, in ? pv : Vb, in);
                pv += n == 1 ? 7 * a.v.tok : a.v.tok;
            }
            if (lane < 2) {  // bytes behind the last key may be anything, 255 (no float's exponent) too: zeros
                const long long e = ((long long)pg * a.H_kv + w.hd) * a.page_size + in0;
                const uint8_t* exps = lane ? a.v_exp : a.k_exp;
                cp_async16(dst + kEOff + lane * 16, pg < a.pages ? exps + e : exps, (uint32_t)min(max(left, 0), 16));
            }
        };
        float o[CH][4];
#pragma unroll
        for (int f = 0; f < CH; ++f) o[f][0] = o[f][1] = o[f][2] = o[f][3] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        // bit i: the i-th tile from now on has keys; tiles are fetched kStages - 1 ahead
        uint32_t there = 0;
        int next = entry_of(0);
#pragma unroll 1
        for (int i = 0; i < kStages - 1; ++i) {
            const int pg = page_at(next);
            next = entry_of(i + 1);
            if (pg >= 0) {
                fetch(i, pg, i);
                there |= 1u << i;
            }
            cp_async_commit();
        }
        int st = 0;
        for (int j = 0; j < nt; ++j) {
            const int key0 = first + j * KT;
            const bool live = there & 1u;
            cp_async_wait<kStages - 2>();
            __syncwarp();  // also: every lane is done with the stage that is filled next
            const uint8_t* stage = ring_p + st * kB;
            const int fill = st == 0 ? kStages - 1 : st - 1;
            st = st == kStages - 1 ? 0 : st + 1;
            auto refill = [&]() {
                const int jn = j + kStages - 1, pg = page_at(next);
                next = entry_of(jn + 1);
                there >>= 1;
                if (pg >= 0) {
                    fetch(jn, pg, fill);
                    there |= 1u << (kStages - 2);
                }
                cp_async_commit();
            };
            if (!live) {
                refill();
                continue;
            }
            // ---- scores of 16 rows and 16 keys
            float c[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) c[i][0] = c[i][1] = c[i][2] = c[i][3] = 0.f;
#pragma unroll
            for (int x = 0; x < X; ++x) {
                uint32_t kw[2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint4 v = *reinterpret_cast<const uint4*>(stage + (x * 2 + i) * 512 + lane * 16);
                    kw[i][0] = v.x, kw[i][1] = v.y, kw[i][2] = v.z, kw[i][3] = v.w;
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint4 qw = qr[x * 4 + k];
                    const uint32_t qa[4] = {qw.x, qw.y, qw.z, qw.w};
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t b0, b1;
                        e4m3x4_to_f16(kw[i][k], b0, b1);
                        mma_16816(c[i], qa, b0, b1);
                    }
                }
            }
            refill();  // here, not before the products: 141 us against 152 for the 64 requests above
            // exponents of keys 2t, 2t + 1, 2t + 8, 2t + 9
            const uint16_t* ex = reinterpret_cast<const uint16_t*>(stage + kEOff) + t;
            const uint32_t ek0 = ex[0] | (uint32_t)ex[4] << 16;
            uint32_t ev0 = ex[8] | (uint32_t)ex[12] << 16;
            // an exponent 0 comes with zeros alone: the smallest there is, for a larger one would lift m above
            // the keys whose values count and cost their P' its bits
            ev0 |= __vcmpeq4(ev0, 0u) & (kMinExp * 0x01010101u);
            // ---- weights.  c[i][2h + b]: row q + 8h, key 8i + 2t + b
            {
                const bool full = key0 >= all_lo && key0 + 16 <= all_hi;
                float y[2][4];
                bool grow = false;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int h = e >> 1, b = e & 1, n = 2 * i + b;
                        y[i][e] = fmaf(c[i][e], rs[h] * up2(ek0, n), minus127(ev0, n));
                        if (!full) {
                            const int key = key0 + 8 * i + 2 * t + b, r = q + 8 * h, p = w.t.pos0 + r / g;
                            bool vis = key < w.t.S_k && r < rows && key_visible(p, key, a.causal, a.window);
                            if (kTree && vis && key >= ctx) vis = tree_sees(a, w.t.q_tok + r / g, key - ctx);
                            y[i][e] = vis ? y[i][e] : -INFINITY;
                        }
                        grow |= y[i][e] > m[h] + kRoom;
                    }
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float mx = quad_max(fmaxf(fmaxf(y[0][2 * h], y[0][2 * h + 1]), fmaxf(y[1][2 * h], y[1][2 * h + 1]))) - kLift;
                        if (mx > m[h]) {
                            const float alpha = m[h] == -INFINITY ? 0.f : ptx::ex2(m[h] - mx);
                            m[h] = mx;
                            l[h] *= alpha;
#pragma unroll
                            for (int f = 0; f < CH; ++f) o[f][2 * h] *= alpha, o[f][2 * h + 1] *= alpha;
                        }
                    }
                }
                const float use[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
                uint32_t pa[4];
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float p0 = ptx::ex2(y[i][2 * h] - use[h]), p1 = ptx::ex2(y[i][2 * h + 1] - use[h]);
                        l[h] = fmaf(p0, down2(ev0, 2 * i), fmaf(p1, down2(ev0, 2 * i + 1), l[h]));
                        pa[2 * i + h] = pack_half2(p0, p1);
                    }
                // ---- P' V
                uint32_t vw[4][CH / 4];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const uint8_t* p = stage + kVOff + (n * 32 + lane) * CH;
                    if constexpr (CH == 16) {
                        const uint4 v = *reinterpret_cast<const uint4*>(p);
                        vw[n][0] = v.x, vw[n][1] = v.y, vw[n][2] = v.z, vw[n][3] = v.w;
                    } else {
                        const uint2 v = *reinterpret_cast<const uint2*>(p);
                        vw[n][0] = v.x, vw[n][1] = v.y;
                    }
                }
#pragma unroll
                for (int f = 0; f < CH; f += 4) {
                    const uint32_t wa = vw[0][f / 4], wb = vw[1][f / 4], wc = vw[2][f / 4], wd = vw[3][f / 4];
                    uint32_t b0, b1, b2, b3;
                    // bytes (a0, b0, a1, b1) and (a2, b2, a3, b3) of two keys' words
                    e4m3x4_to_f16(__byte_perm(wa, wb, 0x5140), b0, b2);
                    e4m3x4_to_f16(__byte_perm(wc, wd, 0x5140), b1, b3);
                    mma_16816(o[f], pa, b0, b1);
                    mma_16816(o[f + 1], pa, b2, b3);
                    e4m3x4_to_f16(__byte_perm(wa, wb, 0x7362), b0, b2);
                    e4m3x4_to_f16(__byte_perm(wc, wd, 0x7362), b1, b3);
                    mma_16816(o[f + 2], pa, b0, b1);
                    mma_16816(o[f + 3], pa, b2, b3);
                }
            }
        }
        // ---- the warps' parts together.  Column n of output tile f is column n CH + f of the head
        cp_async_wait<0>();
        __syncthreads();  // the ring is not in use any more
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float sum = quad_sum(l[h]);
            if (t == 0) s_ml[warp][q + 8 * h] = make_float2(m[h], sum);
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int f = 0; f < CH; f += 4)
                    *reinterpret_cast<float4*>(&s_o[warp][q + 8 * h][(2 * t + b) * CH + f]) =
                        make_float4(o[f][2 * h + b], o[f + 1][2 * h + b], o[f + 2][2 * h + b], o[f + 3][2 * h + b]);
        }
        __syncthreads();
        const bool whole = w.whole();
        const int slot = 2 * (int)blockIdx.x + (w.j0 == 0 ? 1 : 0);
        for (int e = tid; e < rows * (D / 4); e += kThreads) {
            const int r = e / (D / 4), c4 = e % (D / 4) * 4;
            float M = -INFINITY;
#pragma unroll
            for (int v = 0; v < kWarps; ++v) M = fmaxf(M, s_ml[v][r].x);
            const float base = M == -INFINITY ? 0.f : M;
            float L = 0.f;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int v = 0; v < kWarps; ++v) {
                const float2 ml = s_ml[v][r];
                const float f = ptx::ex2(ml.x - base);
                const float4 x = *reinterpret_cast<const float4*>(&s_o[v][r][c4]);
                L = fmaf(ml.y, f, L);
                s.x = fmaf(x.x, f, s.x), s.y = fmaf(x.y, f, s.y), s.z = fmaf(x.z, f, s.z), s.w = fmaf(x.w, f, s.w);
            }
            const int tok = w.t.q_tok + r / g, head = head0 + r % g;
            if (whole) {
                if (c4 == 0) a.LSE[(size_t)head * a.T_q + tok] = lse_of(M, L);
                if (c4 >= a.d) continue;
                const float inv = inv_sum(L);
                const bool none = L == 0.f;  // 0 times a NaN in V is no 0
                alignas(8) T out[4] = {TypeTraits<T>::from_f32(none ? 0.f : s.x * inv), TypeTraits<T>::from_f32(none ? 0.f : s.y * inv),
                                       TypeTraits<T>::from_f32(none ? 0.f : s.z * inv), TypeTraits<T>::from_f32(none ? 0.f : s.w * inv)};
                *reinterpret_cast<uint2*>(static_cast<T*>(a.O) + (long long)tok * a.o.tok + (long long)head * a.o.head + c4) =
                    *reinterpret_cast<const uint2*>(out);
            } else {
                *reinterpret_cast<float4*>(plan.part_o + ((size_t)slot * RT + r) * D + c4) = s;
                if (c4 == 0) plan.part_ml[(size_t)slot * RT + r] = make_float2(part_max(M, L), L);
            }
        }
        __syncthreads();  // nor are the accumulators
        if (!whole) {  // the last part to arrive joins the item
            int first_cta, count;
            w.parts(first_cta, count);
            __threadfence();
            __syncthreads();
            if (tid == 0) s_last = arrive_part(&plan.done[first_cta], plan.tag, count);
            __syncthreads();
            if (s_last) {
                __threadfence();
                join_rows<T, D, kWarps>(a, plan, w.t, head0, g, rows, first_cta, count, s_o, s_row);
            }
        }
    }
}

template <typename T, int D, bool kTree, int kWarps, int kCtas, int kStages>
cudaError_t launch_t(const PackedFwd& a, void* ws, size_t* bytes, cudaStream_t st) {
    const int g = a.H / a.H_kv;
    FwdGeom geo;
    geo.rows = RT;
    geo.tpt = RT / g;
    geo.bn = 16 * kWarps;
    geo.heads = a.H_kv;
    geo.ctas = sm_count() * kCtas;
    geo.D = D;
    geo.min_chunk = kWarps == kManyWarps ? 4 : 2;
    geo.overhead = kWarps == kManyWarps ? 4 : 2;  // filling the ring and the meeting of the warps
    const long long units = plan_units(a, geo);
    geo.self = units <= kSelfUnits && a.N <= kSelfUnits;
    FwdPlan plan;
    *bytes = fwd_plan_layout(a, geo, ws, &plan);
    if (ws == nullptr) return cudaSuccess;
    plan.tag = next_tag();
    cudaError_t e;
    if (!geo.self && (e = launch_fwd_plan(a, geo, plan, st)) != cudaSuccess) return e;
    auto kern = q8_rows_kernel<T, D, kTree, kWarps, kCtas, kStages>;
    static std::atomic<uint64_t> ready{0};
    if ((e = allow_smem(kern, kSmemB<D, kWarps, kStages>, ready)) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)geo.ctas);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = kSmemB<D, kWarps, kStages>;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a, plan, geo, (int)units);
}

template <typename T, int D, bool kTree>
cudaError_t launch_n(const PackedFwd& a, void* ws, size_t* bytes, cudaStream_t st) {
    // a call of fewer (request, head) pairs than half the SMs cuts each into parts for several CTAs
    if ((long long)a.N * a.H_kv * 2 < sm_count()) return launch_t<T, D, kTree, kFewWarps, kFewCtas, kFewStages>(a, ws, bytes, st);
    return launch_t<T, D, kTree, kManyWarps, kManyCtas, kManyStages>(a, ws, bytes, st);
}

template <typename T>
cudaError_t launch_d(const PackedFwd& a, void* ws, size_t* bytes, cudaStream_t st) {
    if (tc_head_dim(a.d) == 64) return a.tree ? launch_n<T, 64, true>(a, ws, bytes, st) : launch_n<T, 64, false>(a, ws, bytes, st);
    return a.tree ? launch_n<T, 128, true>(a, ws, bytes, st) : launch_n<T, 128, false>(a, ws, bytes, st);
}

}  // namespace

cudaError_t launch_q8_rows(const PackedFwd& a, void* ws, size_t* bytes, cudaStream_t st) {
    return a.dtype == FA_F16 ? launch_d<__half>(a, ws, bytes, st) : launch_d<__nv_bfloat16>(a, ws, bytes, st);
}

}  // namespace fa
