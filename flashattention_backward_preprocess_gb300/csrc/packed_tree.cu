// packed_tree.cu -- the instances of the tensor-core forward (packed_fwd_tc.cuh) for trees of new
// tokens over paged caches of the queries' type.
//
// The masks are looked at in the key tiles that hold new tokens alone: a thread shifts the bits of
// its row's token to its columns (one or two words) and clears the scores without one.  The other
// tiles run as without a tree, so a step costs what a causal one of its size does.
#include "packed_fwd_tc.cuh"

namespace fa {

cudaError_t launch_packed_tree(const PackedFwd& a, void* ws, size_t* bytes, cudaStream_t st) {
    return a.dtype == FA_F16 ? launch_paged<__half, true>(a, ws, bytes, st)
                             : launch_paged<__nv_bfloat16, true>(a, ws, bytes, st);
}

}  // namespace fa
