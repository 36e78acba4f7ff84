// packed_q8.cu -- the instances of the tensor-core forward (packed_fwd_tc.cuh) over 8-bit caches.
#include "packed_fwd_tc.cuh"

namespace fa {
namespace {

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

}  // namespace fa
