// packed_q8.cuh -- the converting warps of the tensor-core forward over an 8-bit cache
// (packed_fwd_tc.cuh, kQ8).
//
// A tile's rows are fetched as e4m3 bytes and made fp16 operands in shared memory, a power of two
// away from their values: with the row's exponent e and the tile's largest, E,
//   K' = number * 2^(e - E),  so K = K' 2^E,  V alike,
// so the softmax needs one factor per tile instead of one per key: 2^E_k goes into the scale of the
// scores, E_v into the exponent of P (P' = P 2^E_v), and the row sum takes 2^-E_v of a tile's sum.
// A number times a power of two is exact in fp16 down to 2^-24, so 2^(e - E) loses nothing from
// 2^-14 on (e4m3 starts at 2^-9).  A tile with an exponent further below its largest ("far") keeps its
// numbers as they are, and the softmax takes each key's own exponents to its score and its P (far_scores,
// far_weights in packed_fwd_tc.cuh): one row far larger than the rest, which may be hidden or without
// weight, would otherwise cost all others their bits.  The 32 trees of packed_q8.cu take 481 us with such
// a row in every tile, 261 without.
// fp16 is the operand type for bf16 queries as well (an e4m3 pair is one conversion away from fp16, five
// instructions from bf16): a row of Q is scaled
// by a power of two to a largest magnitude in [2^14, 2^15), which leaves bf16 numbers exact down to
// 2^-31 of it, and P has 11 bits instead of 8.
//
// Two warps look the rows up (table entry, then exponents), row by row, so any page size will do; four
// warps for K and four for V load the numbers into registers, each piece as soon as the one before it
// in its place is converted, and store the operands.
// Rows that are no key of the request (behind its last, before its window, on no page) are zeros.
// A tile takes about 4500 cycles, of which no unit fills half (the products 1300, conversions 500, shared
// memory's bandwidth 1300): the hand-overs between the roles do, and the kernel's length, of whose 80
// registers a thread 80 to 150 bytes are spilled besides (of 16 cycles between two instructions of a warp 4.9
// are awaited instructions, 4.7 memory).  Staging the numbers in shared memory by asynchronous copies first
// took as long.
#pragma once

#include <cuda_fp16.h>

#include "bounded_wait.cuh"
#include "packed.cuh"

namespace fa {
namespace {

// Words of half a looked-up tile: largest exponents of K and V in the low bytes and the first two bits;
// smallest exponents (of those that are not 0).
constexpr uint32_t kInfoValid = 1u << 16;  // there is such a tile
constexpr uint32_t kInfoFirst = 1u << 17;  // it is the first of its item

constexpr uint32_t kTopFar = 1u << 16;     // with a tile's largest exponents: its keys' own ones are to be taken

constexpr uint32_t kMinExp = 97;  // smallest exponent byte of a row that was written

// 16 bytes that this kernel reads once.
__device__ __forceinline__ uint4 ld_once(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
// Two e4m3 numbers (low half of the word: lower byte first) as fp16.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Row t of the Q tile (128-byte swizzled blocks of 64 bf16 columns) to fp16, scaled; returns the
// inverse of the scale.
template <typename C, int D>
__device__ __forceinline__ float convert_q_row(uint8_t* q, int t) {
    auto piece = [&](int c) {
        return reinterpret_cast<uint4*>(q + (c / 8) * C::kBoxQ_B + t * 128 + ((c & 7) ^ (t & 7)) * 16);
    };
    float most = 0.f;
#pragma unroll 4
    for (int c = 0; c < D / 8; ++c) {
        const uint4 w = *piece(c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = (&w.x)[i];
            const float lo = fabsf(__uint_as_float(x << 16)), hi = fabsf(__uint_as_float(x & 0xffff0000u));
            most = fmaxf(most, lo <= 3.4e38f ? lo : 0.f);
            most = fmaxf(most, hi <= 3.4e38f ? hi : 0.f);
        }
    }
    // most * 2^n in [2^14, 2^15), or n = 100 for rows below 2^-86: its inverse times a key's 2^e (2^-30 at
    // least) is above 2^-149, the smallest float
    const int n = most > 0.f ? min(100, 14 - ((__float_as_int(most) >> 23) - 127)) : 0;
    const float s = __int_as_float((n + 127) << 23);
#pragma unroll 4
    for (int c = 0; c < D / 8; ++c) {
        uint4 w = *piece(c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t x = (&w.x)[i];
            const __half2 h = __floats2half2_rn(__uint_as_float(x << 16) * s, __uint_as_float(x & 0xffff0000u) * s);
            (&w.x)[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *piece(c) = w;
    }
    return __int_as_float((127 - n) << 23);
}

// Shared-memory addresses of the barriers of the rings: the first of each.
template <typename C>
struct Q8Bars {
    uint32_t k_full, k_empty, v_full, v_empty, q_full, q_conv, info;
    __device__ __forceinline__ uint32_t info_full(int s) const { return info + 8u * s; }
    __device__ __forceinline__ uint32_t info_empty(int s) const { return info + 8u * (C::INFO + s); }
};

// The two look-up warps, each for half of the rows of every tile of the CTA's share.  A step publishes
// tile j (where its rows lie, their exponents), finds the rows of tile j + 1 and loads their
// exponents, and loads the table entries of tile j + 2.  A word without the valid bit ends the stream.
template <typename C>
__device__ __forceinline__ void look_up_tiles(const PackedFwd& a, const FwdShare& share, const FwdGeom& geo, uint8_t* smem,
                                              volatile int* abort_flag, const Q8Bars<C>& bars, int half) {
    constexpr int BN = C::BN, HB = BN / 2, R = HB / 32;  // rows of the warp and of a lane
    const int lane = threadIdx.x & 31;
    longlong2* at = reinterpret_cast<longlong2*>(smem + C::OFF_AT) + half * HB;
    uint16_t* exps = reinterpret_cast<uint16_t*>(smem + C::OFF_EXP) + half * HB;
    volatile uint2* words = reinterpret_cast<volatile uint2*>(smem + C::OFF_INFO) + half;
    const int shift = (a.page_size & (a.page_size - 1)) == 0 ? 31 - __clz(a.page_size) : -1;
    FwdWalk w;
    bool more = w.init(share, blockIdx.x, a.H_kv, geo.overhead);
    while (more && w.tiles() == 0) more = w.next();
    int j = more ? w.j0 : 0;
    int entry[R], in[R], hd = 0;  // table entries, and rows in their pages (-1: no key)
    auto entries = [&]() -> uint32_t {
        if (!more) return 0u;
        const int key0 = (w.t.n_first + j) * BN + half * HB + lane;
        // keys before the window of the unit's first row may have lost their pages
        const int k_lo = a.window > 0 ? w.t.pos0 - a.window + 1 : 0;
        const int* row = a.table + (size_t)w.t.n * a.max_pages;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int key = key0 + 32 * i;
            in[i] = -1;
            if (key < w.t.S_k && key >= k_lo) {
                const int e = shift >= 0 ? key >> shift : key / a.page_size;
                in[i] = key - e * a.page_size;
                entry[i] = e < a.max_pages ? row[e] : -1;
            }
        }
        hd = w.hd;
        const uint32_t f = kInfoValid | (j == w.j0 ? kInfoFirst : 0u);
        if (++j == w.j1) {
            do more = w.next();
            while (more && w.tiles() == 0);
            if (more) j = w.j0;
        }
        return f;
    };
    long long ko[R], vo[R];  // -1: zeros
    uint8_t ek[R], ev[R];
    auto rows = [&]() {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            ko[i] = vo[i] = -1;
            ek[i] = ev[i] = 0;
            if (in[i] >= 0) {
                bool bad = false;
                const long long pg = page_checked(entry[i], a.pages, &bad);
                if (bad) {
                    atomicOr(a.err, kErrPage);
                } else {
                    ko[i] = pg * a.k_page + (long long)in[i] * a.k.tok + (long long)hd * a.k.head;
                    vo[i] = pg * a.v_page + (long long)in[i] * a.v.tok + (long long)hd * a.v.head;
                    const long long e = (pg * a.H_kv + hd) * a.page_size + in[i];
                    ek[i] = a.k_exp[e];
                    ev[i] = a.v_exp[e];
                }
            }
        }
    };
    // false after a timeout
    auto publish = [&](int tile, uint32_t flags) {
        const int s = tile % C::INFO;
        if (tile >= C::INFO && !wait_bar_warp(bars.info_empty(s), (tile / C::INFO - 1) & 1, abort_flag, a.err)) return false;
        uint32_t mk = 0, mv = 0, lk = 255, lv = 255;
        if (flags) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                at[s * BN + lane + 32 * i] = make_longlong2(ko[i], vo[i]);
                exps[s * BN + lane + 32 * i] = (uint16_t)(ek[i] | ev[i] << 8);
                mk = max(mk, (uint32_t)ek[i]), mv = max(mv, (uint32_t)ev[i]);
                lk = ek[i] ? min(lk, (uint32_t)ek[i]) : lk;
                lv = ev[i] ? min(lv, (uint32_t)ev[i]) : lv;
            }
            mk = __reduce_max_sync(0xffffffffu, mk), mv = __reduce_max_sync(0xffffffffu, mv);
            lk = __reduce_min_sync(0xffffffffu, lk), lv = __reduce_min_sync(0xffffffffu, lv);
        }
        if (lane == 0) {
            words[s * 2].x = mk | mv << 8 | flags;
            words[s * 2].y = lk | lv << 8;
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(bars.info_full(s));
        return true;
    };
    uint32_t now = entries();
    if (now) rows();
    uint32_t next = entries();
    for (int tile = 0; publish(tile, now) && now; ++tile) {
        if (next) rows();
        now = next;
        next = entries();
    }
}

// The eight converting warps.  A timeout leaves the loop of every warp alike: they share no barrier
// but those with bounded waits.
template <typename C, int D, bool kConvQ>
__device__ __forceinline__ void convert_tiles(const PackedFwd& a, uint8_t* smem, volatile int* abort_flag,
                                              const Q8Bars<C>& bars) {
    constexpr int BN = C::BN;
    constexpr int CPR = D / 16;                       // 16-byte pieces of a row
    constexpr int RSTEP = 128 / CPR, N = BN / RSTEP;  // rows between a thread's pieces, pieces per tile
    static_assert(RSTEP % 8 == 0, "a thread's pieces have the same place in their lines");
    static_assert(C::KST == C::VST, "one number of slots");
    const bool is_v = threadIdx.x >= 20 * 32;
    const int t = threadIdx.x & 127, lane = t & 31;
    const int col = t % CPR, row0 = t / CPR;
    unsigned int* err = a.err;
    const long long* at = reinterpret_cast<const long long*>(smem + C::OFF_AT) + 2 * row0 + (is_v ? 1 : 0);
    const uint16_t* exps = reinterpret_cast<const uint16_t*>(smem + C::OFF_EXP) + row0;
    volatile const uint2* words = reinterpret_cast<volatile const uint2*>(smem + C::OFF_INFO);
    const bool col_live = col * 16 < a.d;  // columns behind the head dimension are zeros
    const char* base = static_cast<const char*>(is_v ? a.V : a.K) + (col_live ? col * 16 : 0);
    const int sh = is_v ? 8 : 0;  // of the exponent bytes
    const uint32_t ring = is_v ? C::OFF_V : C::OFF_K, full = is_v ? bars.v_full : bars.k_full;
    const uint32_t empty = is_v ? bars.v_empty : bars.k_empty;
    // where the first piece's halves go: blocks of 64 columns, 128-byte swizzle.  Eight lanes' stores go
    // to eight different pieces of a line: half of them store the odd half first
    const uint32_t even = (uint32_t)(((col & 3) * 2) ^ (row0 & 7)) * 16;
    const bool odd_first = (col & 4) != 0;
    const uint32_t out0 = (uint32_t)(col / 4) * (BN * 128) + row0 * 128 + (odd_first ? even ^ 16u : even);
    const int other = odd_first ? (int)even - (int)(even ^ 16u) : (int)(even ^ 16u) - (int)even;
    auto load = [&](long long o) {
        uint4 q = make_uint4(0u, 0u, 0u, 0u);
        if (o >= 0 && col_live) q = ld_once(base + o);
        return q;
    };
    // whether tile j is there, once it is known
    auto there = [&](int j) {
        if (!wait_bar_warp(bars.info_full(j % C::INFO), (j / C::INFO) & 1, abort_flag, err)) return false;
        const int s = j % C::INFO;
        return (words[s * 2].x & words[s * 2 + 1].x & kInfoValid) != 0;
    };

    uint4 q[N];
    bool more = there(0);
    if (more) {
#pragma unroll
        for (int i = 0; i < N; ++i) q[i] = load(at[i * RSTEP * 2]);
    }
    int ka = 0;
    for (int jg = 0; more; ++jg) {
        const int s = jg % C::INFO, slot = jg % C::KST;
        const uint32_t w0 = words[s * 2].x, w1 = words[s * 2 + 1].x, l0 = words[s * 2].y, l1 = words[s * 2 + 1].y;
        // the largest exponents, and whether any is far below them (in K or in V: both are left as they are then).  Of a tile of exponents 0, zeros alone,
        // V's is the smallest there is: a larger one would lift the softmax's reference above tiles whose
        // values count and cost their P its bits
        const uint32_t mk = max(w0 & 0xff, w1 & 0xff), mv = max(max(w0 >> 8 & 0xff, w1 >> 8 & 0xff), kMinExp);
        const int largest = (int)(is_v ? mv : mk);
        const bool far = min(l0 & 0xff, l1 & 0xff) + 14 < mk || min(l0 >> 8 & 0xff, l1 >> 8 & 0xff) + 14 < mv;
        if (!is_v && t == 0)
            *reinterpret_cast<volatile uint32_t*>(smem + C::OFF_TOP + (jg & 7) * 4) = mk | mv << 8 | (far ? kTopFar : 0u);
        if (far && !is_v && t < BN)
            reinterpret_cast<uint16_t*>(smem + C::OFF_FAR)[(jg & 7) * BN + t] =
                reinterpret_cast<const uint16_t*>(smem + C::OFF_EXP)[s * BN + t];
        if (kConvQ && !is_v && (w0 & kInfoFirst)) {
            if (!wait_bar_warp(bars.q_full, ka & 1, abort_flag, err)) break;
            reinterpret_cast<float*>(smem + C::OFF_QS)[(ka & 3) * 128 + t] = convert_q_row<C, D>(smem + C::OFF_Q, t);
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bars.q_conv);
            ++ka;
        }
        more = there(jg + 1);
        if (jg >= C::KST && !wait_bar_warp(empty + 8u * slot, (jg / C::KST - 1) & 1, abort_flag, err)) break;
        uint8_t* out = smem + ring + slot * C::kTileKV_B + out0;
        const uint16_t* rows = exps + s * BN;
        const int least = far ? 15 : 1;  // f is 2^by, 2^-14 at least (less than that: zeros); 1 in a far tile
        const long long* from = at + (jg + 1) % C::INFO * BN * 2;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int by = (int)(rows[i * RSTEP] >> sh & 0xff) - largest;  // <= 0
            const uint32_t f = (uint32_t)max(by + 15, least) * 0x04000400u;
            uint32_t h[8];
            e4m3x4_to_f16(q[i].x, h[0], h[1]);
            e4m3x4_to_f16(q[i].y, h[2], h[3]);
            e4m3x4_to_f16(q[i].z, h[4], h[5]);
            e4m3x4_to_f16(q[i].w, h[6], h[7]);
            // the same piece of the next tile
            if (more) q[i] = load(from[i * RSTEP * 2]);
#pragma unroll
            for (int c = 0; c < 8; ++c) h[c] = hmul2(h[c], f);
            const uint4 he = make_uint4(h[0], h[1], h[2], h[3]), ho = make_uint4(h[4], h[5], h[6], h[7]);
            uint8_t* line = out + i * RSTEP * 128;
            *reinterpret_cast<uint4*>(line) = odd_first ? ho : he;
            *reinterpret_cast<uint4*>(line + other) = odd_first ? he : ho;
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            ptx::mbar_arrive(full + 8u * slot);
            ptx::mbar_arrive(bars.info_empty(s));
        }
    }
}

}  // namespace
}  // namespace fa
