// packed_q8.cuh -- the converting warps of the tensor-core forward over an 8-bit cache
// (packed_fwd_tc.cuh, kQ8).
//
// A tile's rows are fetched as e4m3 bytes and made fp16 operands in shared memory, a power of two
// away from their values: with the row's exponent e and the tile's largest, E,
//   K' = number * 2^(e - E),  so K = K' 2^E,  V alike,
// so the softmax needs one factor per tile instead of one per key: 2^E_k goes into the scale of the
// scores, E_v into the exponent of P (P' = P 2^E_v), and the row sum takes 2^-E_v of a tile's sum.
// A number times a power of two is exact in fp16 down to 2^-24, so only rows whose values lie below
// 2^-33 of the tile's largest number lose bits.  fp16 is the operand type for bf16 queries as well
// (an e4m3 pair is one conversion away from fp16, five instructions from bf16): a row of Q is scaled
// by a power of two to a largest magnitude in [2^14, 2^15), which leaves bf16 numbers exact down to
// 2^-31 of it, and P has 11 bits instead of 8.
//
// Every thread fetches, with 16-byte asynchronous copies, the pieces that it will convert, so that
// data needs no barrier; rows are looked up (table entry, then exponent) a tile or two ahead, one
// thread per row, any page size.  Rows that are no key of the request (behind its last, before its
// window, on no page) are filled with zeros.
#pragma once

#include <cuda_fp16.h>

#include "bounded_wait.cuh"
#include "packed.cuh"

namespace fa {
namespace {

constexpr uint32_t kConvBarrierId = 6;  // the four converting warps (packed_fwd_tc.cuh has 1 to 5)

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
// 2^n as two equal halves, n <= 0; 0 below fp16's range.
__device__ __forceinline__ uint32_t half2_pow2(int n) {
    const uint32_t h = n >= -14 ? (uint32_t)(n + 15) << 10 : n >= -24 ? 1u << (n + 24) : 0u;
    return h | (h << 16);
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
    // most * 2^n in [2^14, 2^15); n at most 100 keeps its inverse times a key's 2^e a normal number
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

// What the four converting warps do.  Elements of their stream: K and V of each tile in turn.
// A timeout never leaves the loop, so that no warp is left at the barrier: all waits return at once
// then.
template <typename C, typename T, int D, bool kConvQ>
__device__ __forceinline__ void convert_tiles(const PackedFwd& a, const FwdShare& share, const FwdGeom& geo, uint8_t* smem,
                                              volatile int* abort_flag, uint32_t k_full, uint32_t k_empty, uint32_t v_full,
                                              uint32_t v_empty, uint32_t q_full, uint32_t q_conv) {
    constexpr int BN = C::BN, S8 = C::S8, AHEAD = C::AHEAD;
    constexpr int CPR = D / 16;                    // 16-byte pieces of a row
    constexpr int RSTEP = 128 / CPR, N = BN / RSTEP;  // rows between a thread's pieces, pieces per tile
    const int t = threadIdx.x - 16 * 32, lane = t & 31, warp = t >> 5;
    const int col = t % CPR, row0 = t / CPR;
    const uint32_t sbase = ptx::smem_u32(smem);
    unsigned int* err = a.err;
    longlong2* at = reinterpret_cast<longlong2*>(smem + C::OFF_AT);
    uint16_t* exps = reinterpret_cast<uint16_t*>(smem + C::OFF_EXP);
    uint32_t* part = reinterpret_cast<uint32_t*>(smem + C::OFF_PART);
    const bool col_live = col * 16 < a.d;

    FwdWalk w;
    bool more = w.init(share, blockIdx.x, a.H_kv, geo.overhead);
    while (more && w.tiles() == 0) more = w.next();
    int j = more ? w.j0 : 0;
    // the next tile to look up: this thread's row of it
    int nx_entry = -1, nx_in = -1, nx_hd = 0;
    bool nx_valid = false, nx_first = false;
    auto look_up = [&]() {
        nx_valid = more;
        nx_in = -1;
        if (!more) return;
        const int key = (w.t.n_first + j) * BN + t;
        // keys before the window of the unit's first row may have lost their pages
        const int k_lo = a.window > 0 ? w.t.pos0 - a.window + 1 : 0;
        if (t < BN && key < w.t.S_k && key >= k_lo) {
            const int e = key / a.page_size;
            nx_in = key - e * a.page_size;
            nx_entry = e < a.max_pages ? a.table[(size_t)w.t.n * a.max_pages + e] : -1;
        }
        nx_hd = w.hd;
        nx_first = j == w.j0;
        if (++j == w.j1) {
            do more = w.next();
            while (more && w.tiles() == 0);
            if (more) j = w.j0;
        }
    };
    // exponents (K, V in the next byte) of this thread's row of tiles jg .. jg + AHEAD; whether each
    // is there, and the first of its item
    uint32_t ex[AHEAD + 1];
    uint32_t valid = 0, first = 0;
    // where the rows of the looked-up tile lie, to the others
    auto enter = [&](int tile, int i) {
        longlong2 o = make_longlong2(-1, -1);
        ex[i] = 0;
        if (nx_valid && nx_in >= 0) {
            bool bad = false;
            const long long pg = page_checked(nx_entry, a.pages, &bad);
            if (bad) {
                atomicOr(err, kErrPage);
            } else {
                o.x = pg * a.k_page + (long long)nx_in * a.k.tok + (long long)nx_hd * a.k.head;
                o.y = pg * a.v_page + (long long)nx_in * a.v.tok + (long long)nx_hd * a.v.head;
                const long long e = (pg * a.H_kv + nx_hd) * a.page_size + nx_in;
                ex[i] = a.k_exp[e] | (uint32_t)a.v_exp[e] << 8;
            }
        }
        if (t < BN) at[(tile & 3) * BN + t] = o;
        valid |= (uint32_t)nx_valid << i;
        first |= (uint32_t)(nx_valid && nx_first) << i;
    };
    // fetches element n of the stream (tile n / 2) into its slot
    auto fetch = [&](int n, bool there) {
        if (there && col_live) {
            const char* base = static_cast<const char*>((n & 1) ? a.V : a.K) + col * 16;
            const longlong2* rows = at + ((n >> 1) & 3) * BN;
            const uint32_t dst = sbase + C::OFF_8 + (uint32_t)(n % S8) * C::kTile8_B + t * 16;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const longlong2 o2 = rows[row0 + i * RSTEP];
                const long long o = (n & 1) ? o2.y : o2.x;
                cp_async16(dst + i * 2048, base + (o < 0 ? 0 : o), o < 0 ? 0u : 16u);
            }
        }
        cp_async_commit();
    };
    // makes a fetched tile an operand tile at `dst` (blocks of 64 columns, 128-byte swizzle); `sh`: the
    // byte of the rows' exponents
    auto convert = [&](int n, uint32_t dst, const uint16_t* rows, int sh, int top) {
        const uint32_t src = C::OFF_8 + (uint32_t)(n % S8) * C::kTile8_B + t * 16;
        const uint32_t out = dst + (uint32_t)(col / 4) * (BN * 128);
        const bool odd_first = (col & 4) != 0;  // eight lanes' stores to eight different pieces of a line
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int r = row0 + i * RSTEP;
            const uint4 q = col_live ? *reinterpret_cast<const uint4*>(smem + src + i * 2048) : make_uint4(0u, 0u, 0u, 0u);
            const int by = (int)(rows[r] >> sh & 0xff) - top;  // <= 0
            const uint32_t f = half2_pow2(by < -14 ? -14 : by);
            uint32_t h[8];
#pragma unroll
            for (int c = 0; c < 4; ++c) e4m3x4_to_f16((&q.x)[c], h[2 * c], h[2 * c + 1]);
#pragma unroll
            for (int c = 0; c < 8; ++c) h[c] = hmul2(h[c], f);
            if (by < -14) {
                const uint32_t f2 = half2_pow2(by + 14);
#pragma unroll
                for (int c = 0; c < 8; ++c) h[c] = hmul2(h[c], f2);
            }
            const int c0 = (col & 3) * 2;
            uint8_t* line = smem + out + r * 128;
            uint4* even = reinterpret_cast<uint4*>(line + ((c0 ^ (r & 7)) * 16));
            uint4* odd = reinterpret_cast<uint4*>(line + (((c0 + 1) ^ (r & 7)) * 16));
            const uint4 he = make_uint4(h[0], h[1], h[2], h[3]), ho = make_uint4(h[4], h[5], h[6], h[7]);
            *(odd_first ? odd : even) = odd_first ? ho : he;
            *(odd_first ? even : odd) = odd_first ? he : ho;
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
    };

    look_up();
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
        enter(i, i);
        look_up();
    }
    ex[AHEAD] = 0;
    ptx::named_bar_sync(kConvBarrierId, 128);
#pragma unroll
    for (int n = 0; n < S8; ++n) fetch(n, valid >> (n / 2) & 1u);
    int ka = 0;
    for (int jg = 0; valid & 1u; ++jg) {
        enter(jg + AHEAD, AHEAD);
        look_up();
        // the tile's largest exponents
        const int s2 = jg & 1;
        if (t < BN) exps[s2 * BN + t] = (uint16_t)ex[0];
        const uint32_t mk = __reduce_max_sync(0xffffffffu, ex[0] & 0xffu), mv = __reduce_max_sync(0xffffffffu, ex[0] >> 8);
        if (lane == 0) part[s2 * 4 + warp] = mk | mv << 8;
        __syncwarp();
        ptx::named_bar_sync(kConvBarrierId, 128);
        uint32_t tk = 0, tv = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t p = part[s2 * 4 + i];
            tk = max(tk, p & 0xffu);
            tv = max(tv, p >> 8);
        }
        tv = max(tv, 1u);  // 2^-ev is a number
        if (t == 0) *reinterpret_cast<volatile uint32_t*>(smem + C::OFF_TOP + (jg & 7) * 4) = tk | tv << 8;
        if (first & 1u) {
            if constexpr (kConvQ) {
                wait_bar_warp(q_full, ka & 1, abort_flag, err);
                reinterpret_cast<float*>(smem + C::OFF_QS)[(ka & 3) * 128 + t] = convert_q_row<C, D>(smem + C::OFF_Q, t);
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(q_conv);
            }
            ++ka;
        }
        // K
        cp_async_wait<S8 - 1>();
        const int sk = jg % C::KST, sv = jg % C::VST;
        if (jg >= C::KST) wait_bar_warp(k_empty + 8u * sk, (jg / C::KST - 1) & 1, abort_flag, err);
        convert(2 * jg, C::OFF_K + sk * C::kTileKV_B, exps + s2 * BN, 0, (int)tk);
        if (lane == 0) ptx::mbar_arrive(k_full + 8u * sk);
        fetch(2 * jg + S8, valid >> (S8 / 2) & 1u);
        // V
        cp_async_wait<S8 - 1>();
        if (jg >= C::VST) wait_bar_warp(v_empty + 8u * sv, (jg / C::VST - 1) & 1, abort_flag, err);
        convert(2 * jg + 1, C::OFF_V + sv * C::kTileKV_B, exps + s2 * BN, 8, (int)tv);
        if (lane == 0) ptx::mbar_arrive(v_full + 8u * sv);
        fetch(2 * jg + 1 + S8, valid >> ((S8 + 1) / 2) & 1u);
        valid >>= 1;
        first >>= 1;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) ex[i] = ex[i + 1];
    }
    cp_async_wait<0>();
}

}  // namespace
}  // namespace fa
