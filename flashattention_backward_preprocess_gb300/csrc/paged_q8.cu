// paged_q8.cu -- an 8-bit key/value cache: rows quantised as they are written, and read back.
//
// A row (one token and head of K or V, d elements) is d e4m3 numbers q and one exponent byte b:
//   e = the smallest whole number with max |x| <= 448 * 2^e, kept in [lo, hi];  b = e + 127
//   q = x * 2^-e rounded to e4m3 (to nearest, halves to even);  the value is q * 2^e
// A power of two as the scale makes x * 2^-e exact, so every element is rounded once, by at most
// 2^-4 of itself (or 2^-10 * 2^e where that is more), and reading a value back rounds nothing:
// four significant bits fit every type.  max / 448 as the scale would be no nearer: e4m3 is a
// floating-point type, whose step follows the value.
//   lo, hi = -30, 30 (fp32, bf16): rows below 448 * 2^-30 have a fixed step of 2^-39, values above
//            448 * 2^30 stay there;  -15, 8 (fp16): steps of 2^-24, fp16's own, and values above
//            61440 stay there, since the next e4m3 number is past fp16's range.
// Infinities and NaN are stored as NaN and leave the exponent to the row's other elements.
//
// A group of lanes holds a row, 16 elements a lane: loads of 32 or 64 bytes, the max over the group
// by shuffles, a store of 16 bytes.  K and V of a row belong to the same lanes, so both loads are in
// flight together.  Bound by DRAM: 16384 tokens of H_kv = 8, d = 128, bf16 (101 MB) take 24 us to write
// (4.2 TB/s) and 15 to read back (6.7 TB/s).
#include <cuda_fp8.h>

#include "packed.cuh"
#include "paged_cache.cuh"

namespace fa {
namespace {

constexpr int kT = 256;

template <typename T>
struct Q8Limits {
    static constexpr int kLo = -30, kHi = 30;
    static constexpr float kMost = 448.f * 1073741824.f;
};
template <>
struct Q8Limits<__half> {
    static constexpr int kLo = -15, kHi = 8;
    static constexpr float kMost = 61440.f;
};

// 64-bit divisions take a hundred instructions: pages of a power of two of rows are shifted, and item
// numbers below 2^32 divided as such.
struct Page {
    long long pg, row;
};
__device__ __forceinline__ Page page_row(long long slot, int page_size) {
    if (slot < 0) return {0, slot};
    if ((page_size & (page_size - 1)) == 0) return {slot >> (31 - __clz(page_size)), slot & (page_size - 1)};
    const long long pg = slot / page_size;
    return {pg, slot - pg * page_size};
}
__device__ __forceinline__ int quotient(long long i, int n, bool small) {
    return small ? (int)((unsigned)i / (unsigned)n) : (int)(i / n);
}

// Sixteen elements from p (16-byte aligned) as fp32.
template <typename T>
__device__ __forceinline__ void load16(const char* p, float* x) {
    constexpr int kWords = 16 * (int)sizeof(T) / 16, kPer = 16 / (int)sizeof(T);
    uint4 w[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
#pragma unroll
    for (int i = 0; i < kWords; ++i)
#pragma unroll
        for (int c = 0; c < kPer; ++c) x[i * kPer + c] = TypeTraits<T>::to_f32(reinterpret_cast<const T*>(&w[i])[c]);
}

// Largest finite magnitude.
__device__ __forceinline__ float most16(const float* x) {
    float m = 0.f;
#pragma unroll
    for (int c = 0; c < 16; ++c) m = fmaxf(m, fabsf(x[c]) <= 3.402823466e38f ? fabsf(x[c]) : 0.f);
    return m;
}

// Smallest e with m <= 448 * 2^e, within the limits.  448 = 1.75 * 2^8.
template <typename T>
__device__ __forceinline__ int exponent(float m) {
    const int b = __float_as_int(m);
    const int e = (b >> 23) - 127 - 8 + ((b & 0x7fffff) > 0x600000);
    return max(Q8Limits<T>::kLo, min(Q8Limits<T>::kHi, e));
}

template <typename T>
__device__ __forceinline__ uint4 numbers(const float* x, int e) {
    const float s = __int_as_float((127 - e) << 23);  // 2^-e
    constexpr float most = Q8Limits<T>::kMost;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int c = 0; c < 16; c += 2) {
        float y[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float v = x[c + i];
            y[i] = fabsf(v) <= 3.402823466e38f ? fminf(fmaxf(v, -most), most) * s : __int_as_float(0x7fffffff);
        }
        const uint32_t pair = __nv_cvt_float2_to_fp8x2(make_float2(y[0], y[1]), __NV_SATFINITE, __NV_E4M3);
        w[c / 4] |= pair << (c % 4 * 8);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// kLanes: lanes of a row, d / 16 rounded up to a power of two.
template <typename T, int kLanes>
__global__ void __launch_bounds__(kT) paged_write_q8_kernel(const PagedQ8 a) {
    const int x = threadIdx.x % kLanes;
    const long long total = (long long)a.T * a.H_kv, step = (long long)gridDim.x * (kT / kLanes);
    const bool live = x * 16 < a.d;
    // whole warps walk together: the max of a row is a shuffle
    for (long long r0 = (long long)blockIdx.x * (kT / kLanes) + threadIdx.x / 32 * (32 / kLanes); r0 < total; r0 += step) {
        const long long r = r0 + threadIdx.x % 32 / kLanes;
        const long long rc = min(r, total - 1);
        const int t = quotient(rc, a.H_kv, total < (1ll << 32)), h = (int)(rc - (long long)t * a.H_kv);
        const long long slot = a.slots[t];
        const auto [pg, row] = page_row(slot, a.page_size);
        const bool in = r < total && slot >= 0 && pg < a.pages;
        if (r < total && slot >= 0 && !in && x == 0 && h == 0) atomicOr(a.err, kErrPage);
        float k[16], v[16], mk = 0.f, mv = 0.f;
        if (in && live) {
            load16<T>(static_cast<const char*>(a.K) + t * a.k.tok + h * a.k.head + x * 16 * (int)sizeof(T), k);
            load16<T>(static_cast<const char*>(a.V) + t * a.v.tok + h * a.v.head + x * 16 * (int)sizeof(T), v);
            mk = most16(k);
            mv = most16(v);
        }
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) {
            mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, o));
            mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, o));
        }
        if (!in || !live) continue;
        const int ek = exponent<T>(mk), ev = exponent<T>(mv);
        *reinterpret_cast<uint4*>(static_cast<char*>(a.K_cache) + pg * a.kc_page + row * a.kc.tok + h * a.kc.head + x * 16) =
            numbers<T>(k, ek);
        *reinterpret_cast<uint4*>(static_cast<char*>(a.V_cache) + pg * a.vc_page + row * a.vc.tok + h * a.vc.head + x * 16) =
            numbers<T>(v, ev);
        if (x == 0) {
            const long long at = (pg * a.H_kv + h) * a.page_size + row;
            a.k_exp[at] = (uint8_t)(ek + 127);
            a.v_exp[at] = (uint8_t)(ev + 127);
        }
    }
}

// Sixteen values q * 2^e to p, in T.
template <typename T>
__device__ __forceinline__ void store16(char* p, uint4 q, float s) {
    constexpr int kWords = 16 * (int)sizeof(T) / 16, kPer = 16 / (int)sizeof(T);
    uint4 w[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i)
#pragma unroll
        for (int c = 0; c < kPer; ++c) {
            const int n = i * kPer + c;
            __nv_fp8_e4m3 b;
            b.__x = (__nv_fp8_storage_t)((&q.x)[n / 4] >> (n % 4 * 8));
            reinterpret_cast<T*>(&w[i])[c] = TypeTraits<T>::from_f32(static_cast<float>(b) * s);
        }
#pragma unroll
    for (int i = 0; i < kWords; ++i) __stcs(reinterpret_cast<uint4*>(p) + i, w[i]);
}

template <typename T>
__global__ void __launch_bounds__(kT) paged_read_q8_kernel(const PagedQ8 a) {
    const int cpr = a.d / 16, per = a.H_kv * cpr;
    const long long total = (long long)a.T * per, step = (long long)gridDim.x * kT;
    for (long long i = (long long)blockIdx.x * kT + threadIdx.x; i < total; i += step) {
        const int t = quotient(i, per, total < (1ll << 32)), c = (int)(i - (long long)t * per);
        const int h = c / cpr, x = c - h * cpr;
        const long long slot = a.slots[t];
        const auto [pg, row] = page_row(slot, a.page_size);
        uint4 k = make_uint4(0u, 0u, 0u, 0u), v = k;
        float sk = 0.f, sv = 0.f;
        if (slot >= 0 && pg < a.pages) {
            const long long at = (pg * a.H_kv + h) * a.page_size + row;
            k = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.K_cache) + pg * a.kc_page + row * a.kc.tok + h * a.kc.head + x * 16);
            v = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.V_cache) + pg * a.vc_page + row * a.vc.tok + h * a.vc.head + x * 16);
            sk = exp_value(a.k_exp[at]);
            sv = exp_value(a.v_exp[at]);
        } else if (slot >= 0 && c == 0) {
            atomicOr(a.err, kErrPage);
        }
        store16<T>(static_cast<char*>(a.K) + t * a.k.tok + h * a.k.head + x * 16 * (int)sizeof(T), k, sk);
        store16<T>(static_cast<char*>(a.V) + t * a.v.tok + h * a.v.head + x * 16 * (int)sizeof(T), v, sv);
    }
}

unsigned grid_for(long long items, int per_block) {
    const long long n = (items + per_block - 1) / per_block;
    return (unsigned)(n > 152 * 32 ? 152 * 32 : n);
}

template <typename T, int kLanes>
cudaError_t write_t(const PagedQ8& a, cudaStream_t st) {
    paged_write_q8_kernel<T, kLanes><<<grid_for((long long)a.T * a.H_kv, kT / kLanes), kT, 0, st>>>(a);
    return cudaGetLastError();
}
template <typename T>
cudaError_t write_d(const PagedQ8& a, cudaStream_t st) {
    if (a.d <= 32) return write_t<T, 2>(a, st);
    if (a.d <= 64) return write_t<T, 4>(a, st);
    if (a.d <= 128) return write_t<T, 8>(a, st);
    return write_t<T, 16>(a, st);
}
template <typename T>
cudaError_t read_t(const PagedQ8& a, cudaStream_t st) {
    paged_read_q8_kernel<T><<<grid_for((long long)a.T * a.H_kv * (a.d / 16), kT), kT, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_write_q8(const PagedQ8& a, cudaStream_t st) {
    if (a.dtype == FA_F32) return write_d<float>(a, st);
    return a.dtype == FA_F16 ? write_d<__half>(a, st) : write_d<__nv_bfloat16>(a, st);
}
cudaError_t launch_paged_read_q8(const PagedQ8& a, cudaStream_t st) {
    if (a.dtype == FA_F32) return read_t<float>(a, st);
    return a.dtype == FA_F16 ? read_t<__half>(a, st) : read_t<__nv_bfloat16>(a, st);
}

}  // namespace fa
