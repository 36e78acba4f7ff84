// paged_cache.cuh -- arguments of the paged-cache bookkeeping and write kernels.
#pragma once

#include "packed.cuh"

namespace fa {

struct PageSlots {
    const int *ctx_lens, *cu_q, *free_pages, *free_start;
    int* table;  // [N, max_pages], columns of new pages written
    long long* slots;
    int *positions, *seq_lens, *free_next;
    int N, T, n_free, page_size, max_pages;
    unsigned int* err;
};
cudaError_t launch_page_slots(const PageSlots& a, cudaStream_t st);

// Strides in bytes.
struct PagedWrite {
    const void *K, *V;
    void *K_cache, *V_cache;
    const long long* slots;
    int T, H_kv, cpr;  // cpr: 16-byte pieces of one head's row
    int pages, page_size;
    RowStride k, v, kc, vc;
    long long kc_page, vc_page;
    unsigned int* err;
};
cudaError_t launch_paged_write(const PagedWrite& a, cudaStream_t st);

}  // namespace fa
