// packed_q8.cu -- the instances of the tensor-core forward (packed_fwd_tc.cuh) over 8-bit caches, and
// the way round them for calls of many rows.
//
// In the tensor-core kernel every 128-row tile of a request converts the request's keys again, and the
// conversion is what takes its time (about 4500 cycles of a 128-key tile; the products need 1300).
// Where requests have many such tiles (chunks of prompts), one pass makes the rows of the cache that
// the step reads fp16 or bf16, exactly, in pages of the workspace, and the kernel for caches of that
// type does the rest.  10 chunks of up to 512 tokens over up to 8000 cached ones, H = 32, H_kv = 8, d = 128,
// bf16: 157 us (42 of them the copy of 54 MB) against 316.  32 trees of 8 to 64 tokens over 100 to 6000,
// f16, in the converting kernel: 256 us; the copy alone would write 400 MB.
//
// Every number that fa_paged_write_q8 stores is a bf16 number; fp16 holds those written from fp16.  A row that
// it cannot hold is noticed by the copy, and the converting kernel does the step instead: one more
// launch for fp16, 173 us in place of 162 for the ten chunks.
//
// A bf16 row's P has 8 bits behind the copy and 11 in the other two kernels, so a request's result may differ by
// such roundings with the requests that share its call.
#include "packed_fwd_tc.cuh"

namespace fa {
namespace {

constexpr int kSpreadT = 256, kSpreadTok = 32;  // threads of a block, tokens

// Tokens [kSpreadTok * blockIdx.x, ..) of request blockIdx.y, those that its new tokens may see, to pages
// of its own: entry e of its table becomes page max_pages * n + e.
// fp16: rows of a cache that was written from a wider type may not fit.  *wide is set then (it was 0 before).
template <typename T>
__global__ void __launch_bounds__(kSpreadT) q8_spread_kernel(const PackedFwd a, T* K, T* V, int* table, unsigned int* wide) {
    constexpr bool kHalf = TypeTraits<T>::kId == FA_F16;
    bool lost = false;
    const int n = blockIdx.y, k0 = blockIdx.x * kSpreadTok;
    Seq s;
    if (!seq_at(a, n, s) || s.nq == 0) return;  // the plan reports lengths that do not fit
    for (int e = k0 / a.page_size + threadIdx.x; e < a.max_pages && (long long)e * a.page_size < k0 + kSpreadTok; e += kSpreadT)
        if ((long long)e * a.page_size >= k0) table[(size_t)n * a.max_pages + e] = n * a.max_pages + e;
    // whole pages from the first key that any new token sees: none of their rows may be left unset
    int lo = a.window > 0 ? max(s.nk - s.nq - a.window + 1, 0) : 0;
    lo -= lo % a.page_size;
    const int hi = (int)min((long long)s.nk, table_room(a));
    const int per = a.H_kv * (a.d / 16);
    for (int i = threadIdx.x; i < kSpreadTok * per; i += kSpreadT) {
        const int j = k0 + i / per, c = i % per, h = c / (a.d / 16), x = c % (a.d / 16) * 16;
        if (j < lo || j >= hi) continue;
        const int in = j % a.page_size;
        bool bad = false;
        const long long pg = page_of(a.table + (size_t)n * a.max_pages, j, a.page_size, a.max_pages, a.pages, &bad);
        uint4 k = make_uint4(0u, 0u, 0u, 0u), v = k;
        float sk = 0.f, sv = 0.f;
        if (bad) {
            if (c == 0) atomicOr(a.err, kErrPage);
        } else {
            k = ld_once(static_cast<const char*>(a.K) + pg * a.k_page + in * a.k.tok + h * a.k.head + x);
            v = ld_once(static_cast<const char*>(a.V) + pg * a.v_page + in * a.v.tok + h * a.v.head + x);
            const long long e = (pg * a.H_kv + h) * a.page_size + in;
            const uint8_t ek = a.k_exp[e], ev = a.v_exp[e];
            sk = exp_value(ek);
            sv = exp_value(ev);
            // numbers are multiples of 2^-9, fp16's of 2^-24
            if (kHalf) lost |= (ek != 0 && ek < 127 - 15) || (ev != 0 && ev < 127 - 15);
        }
        const long long to = (((long long)n * a.max_pages * a.page_size + j) * a.H_kv + h) * a.d + x;
        auto put = [&](T* dst, const uint4& q, float f) {
            uint32_t w[8];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                uint32_t lo2, hi2;
                e4m3x4_to_f16((&q.x)[u], lo2, hi2);
                const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&lo2));
                const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&hi2));
                if (kHalf) lost |= fmaxf(fmaxf(fabsf(p.x), fabsf(p.y)), fmaxf(fabsf(r.x), fabsf(r.y))) * f > 65504.f;
                w[2 * u] = pack2<TypeTraits<T>::kId == FA_BF16>(p.x * f, p.y * f);
                w[2 * u + 1] = pack2<TypeTraits<T>::kId == FA_BF16>(r.x * f, r.y * f);
            }
            reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
            reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
        };
        put(K + to, k, sk);
        put(V + to, v, sv);
    }
    if (kHalf && lost) *wide = 1u;
}

size_t spread_cache_bytes(const PackedFwd& a) {
    return packed_align((size_t)a.N * a.max_pages * a.page_size * a.H_kv * a.d * 2);
}
size_t spread_table_bytes(const PackedFwd& a) { return packed_align((size_t)a.N * a.max_pages * 4); }
constexpr size_t kSpreadWordBytes = 256;  // the word `wide`

template <typename T, bool kTree>
cudaError_t launch_d(const PackedFwd& a, void* ws, size_t* bytes, cudaStream_t st) {
    const int D = a.d == 256 ? 256 : tc_head_dim(a.d);
    if (D == 64) return launch_t<T, 64, true, false, kTree, true>(a, ws, bytes, st);
    if (D == 128) return launch_t<T, 128, true, false, kTree, true>(a, ws, bytes, st);
    if (D == 256) return launch_t<T, 256, true, false, kTree, true>(a, ws, bytes, st);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_packed_q8(const PackedFwd& a, void* ws, size_t* bytes, cudaStream_t st) {
    if (a.dtype == FA_F16) return a.tree ? launch_d<__half, true>(a, ws, bytes, st) : launch_d<__half, false>(a, ws, bytes, st);
    return a.tree ? launch_d<__nv_bfloat16, true>(a, ws, bytes, st) : launch_d<__nv_bfloat16, false>(a, ws, bytes, st);
}

// From four 128-row tiles per request on, where the copy (of all that the tables have room for: the
// lengths are on the device) takes 2 GB each of K and V at most, and pages that the other kernel takes.
// Eight requests of 256, 384, 512, 768 and 1024 rows over 500 to 8000 keys, H_kv = 8, us in a replayed graph:
//   bf16, d = 128   copied 146, 155, 185, 203, 241   converted in tiles 140, 186, 238, 337, 435
//   f16,  d = 128          164, 164, 195, 212, 255                      129, 166, 211, 296, 382
//   bf16, d = 64            89, 101, 117, 146, 176                      113, 150, 191, 272, 354
// so the copy is even at about 300 rows; below 512 it would save a sixth at most (a third at d = 64), for a
// workspace larger than the cache itself.
bool q8_spread(const PackedFwd& a) {
    const long long g = a.H / a.H_kv;
    const int bn = a.d == 256 ? 64 : 128;
    const bool pages = a.page_size % 8 == 0 && (bn % a.page_size == 0 || a.page_size % bn == 0);
    return pages && a.T_q * g >= 512ll * a.N && a.N <= 65535 &&
           (double)a.N * a.max_pages * a.page_size * a.H_kv * a.d * 2 <= 2147483648.0;
}

cudaError_t launch_q8_spread(const PackedFwd& a, void* ws, size_t* bytes, cudaStream_t st) {
    const size_t cache = spread_cache_bytes(a), table = spread_table_bytes(a);
    char* base = static_cast<char*>(ws);
    PackedFwd b = a;
    b.k_exp = b.v_exp = nullptr;
    b.pages = a.N * a.max_pages;
    b.k.head = b.v.head = a.d;
    b.k.tok = b.v.tok = (long long)a.H_kv * a.d;
    b.k_page = b.v_page = b.k.tok * a.page_size;
    if (ws == nullptr) {
        cudaError_t e = launch_packed_fwd(b, nullptr, bytes, st);
        if (a.dtype == FA_F16) {
            size_t other = 0;
            if (e == cudaSuccess) e = launch_packed_q8(a, nullptr, &other, st);
            *bytes = *bytes > other ? *bytes : other;
        }
        *bytes += 2 * cache + table + kSpreadWordBytes;
        return e;
    }
    b.K = base, b.V = base + cache;
    int* own = reinterpret_cast<int*>(base + 2 * cache);
    b.table = own;
    unsigned int* wide = reinterpret_cast<unsigned int*>(base + 2 * cache + table);
    char* rest = base + 2 * cache + table + kSpreadWordBytes;
    const long long room = (long long)a.max_pages * a.page_size;
    const dim3 grid((unsigned)((room + kSpreadTok - 1) / kSpreadTok), (unsigned)a.N);
    cudaError_t e;
    if (a.dtype == FA_F16) {
        if ((e = cudaMemsetAsync(wide, 0, sizeof(unsigned int), st)) != cudaSuccess) return e;
        q8_spread_kernel<<<grid, kSpreadT, 0, st>>>(a, reinterpret_cast<__half*>(base), reinterpret_cast<__half*>(base + cache), own, wide);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        // of the two kernels one finds nothing to do; they follow each other, so the scratch is one
        PackedFwd c = a;
        b.gate = c.gate = wide;
        b.gate_value = 0u, c.gate_value = 1u;
        if ((e = launch_packed_fwd(b, rest, bytes, st)) != cudaSuccess) return e;
        return launch_packed_q8(c, rest, bytes, st);
    }
    q8_spread_kernel<<<grid, kSpreadT, 0, st>>>(a, reinterpret_cast<__nv_bfloat16*>(base),
                                                reinterpret_cast<__nv_bfloat16*>(base + cache), own, wide);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_packed_fwd(b, rest, bytes, st);
}

}  // namespace fa
