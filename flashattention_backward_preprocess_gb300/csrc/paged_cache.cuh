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

// Rows of an 8-bit cache: written from K, V (elements of `dtype`) or read back into them.
// Strides in bytes; exponents dense [pages, H_kv, page_size].
struct PagedQ8 {
    void *K, *V;
    void *K_cache, *V_cache;
    uint8_t *k_exp, *v_exp;
    const long long* slots;
    int T, H_kv, d, pages, page_size, dtype;
    RowStride k, v, kc, vc;
    long long kc_page, vc_page;
    unsigned int* err;
};
cudaError_t launch_paged_write_q8(const PagedQ8& a, cudaStream_t st);
cudaError_t launch_paged_read_q8(const PagedQ8& a, cudaStream_t st);

// Ancestor masks and positions of the new tokens.
struct TreeMask {
    const int *parents, *cu_q, *ctx_lens;
    unsigned long long* tree;  // [T, words]
    int* positions;            // [T]
    int N, T, words;
    unsigned int* err;
};
cudaError_t launch_tree_mask(const TreeMask& a, cudaStream_t st);

// Rows of the accepted tokens moved up, in the caches of up to kKeepLayers layers.  Strides in bytes.
constexpr int kKeepLayers = 32;
struct PagedKeep {
    void *K[kKeepLayers], *V[kKeepLayers];
    uint8_t *k_exp[kKeepLayers], *v_exp[kKeepLayers];  // null: not an 8-bit cache
    const int *path, *count, *cu_q, *seq_lens, *table;
    int layers, N, T, H_kv, cpr;  // cpr: 16-byte pieces of one head's row
    int pages, page_size, max_pages;
    RowStride kc, vc;
    long long kc_page, vc_page;
    unsigned int* err;
};
cudaError_t launch_paged_keep(const PagedKeep& a, cudaStream_t st);

// Lengths after the step and the pages behind them.
struct PageTrim {
    bool by_path;     // a request that PagedKeep leaves alone keeps all tokens, the others do not mind it
    const int* path;  // then, [T] as in PagedKeep
    const int *count, *cu_q, *seq_lens, *table, *free_start;
    int *free_pages, *lens, *free_next;
    int N, T, n_free, page_size, max_pages;
    unsigned int* err;
};
cudaError_t launch_page_trim(const PageTrim& a, cudaStream_t st);

}  // namespace fa
