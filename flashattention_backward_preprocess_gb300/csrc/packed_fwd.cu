// packed_fwd.cu -- the instances of the tensor-core forward (packed_fwd_tc.cuh) for packed
// sequences and for paged caches of the queries' type.
#include "packed_fwd_tc.cuh"

namespace fa {
namespace {

// Steps over an 8-bit cache whose requests have 32 rows (tokens x heads of a group) or fewer on
// average, idle ones counted too, on pages of whole 16-key pieces: packed_q8_rows.cu, which reads the cache
// once per 16 rows.  32 requests of 8, 16, 32, 48 and 64 rows over 98000 keys, bf16, us in a replayed graph:
//   d = 128, H_kv = 8, 4 heads a group (1 and 8: the same)   there 78, 81, 130, 179, 226
//                                                            in 128-row tiles 147, 148, 154, 158, 171
//   d = 64, H_kv = 8, 4 heads    57, 58, 91, 124, 156        119, 120, 124, 128, 134
//   d = 128, H_kv = 2, 16 heads      48, 66, 86, 105              58, 62, 65, 70
bool few_rows(const PackedFwd& a) {
    const long long g = a.H / a.H_kv;
    return a.d <= 128 && g <= 16 && a.page_size % 16 == 0 && a.T_q * g <= 32ll * a.N;
}

template <typename T>
cudaError_t launch_d(const PackedFwd& a, void* ws, size_t* bytes, cudaStream_t st) {
    if (a.paged()) return launch_paged<T, false>(a, ws, bytes, st);
    const int D = a.d == 256 ? 256 : tc_head_dim(a.d);
    if (D == 64) return launch_t<T, 64, false, false, false>(a, ws, bytes, st);
    if (D == 128) return launch_t<T, 128, false, false, false>(a, ws, bytes, st);
    if (D == 256) return launch_t<T, 256, false, false, false>(a, ws, bytes, st);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_packed_fwd(const PackedFwd& a, void* ws, size_t* bytes, cudaStream_t st) {
    if (a.q8() && few_rows(a)) return launch_q8_rows(a, ws, bytes, st);
    if (a.q8() && q8_spread(a)) return launch_q8_spread(a, ws, bytes, st);
    if (a.q8()) return launch_packed_q8(a, ws, bytes, st);
    if (a.tree) return launch_packed_tree(a, ws, bytes, st);
    return a.dtype == FA_F16 ? launch_d<__half>(a, ws, bytes, st) : launch_d<__nv_bfloat16>(a, ws, bytes, st);
}

}  // namespace fa
