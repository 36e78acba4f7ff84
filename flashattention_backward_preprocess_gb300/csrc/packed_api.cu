// packed_api.cu -- C entry points of the packed and paged attention operators (include/fa.h):
// argument checks, the choice of kernel, and the device word in which their kernels record
// what only the device can see (lengths, pages, timeouts).
#include <math.h>
#include <time.h>

#include <algorithm>
#include <mutex>
#include <new>
#include <string>
#include <vector>

#include "packed.cuh"
#include "paged_cache.cuh"

namespace {
constexpr int kMaxDevices = 64;
}

// Error word of the packed and paged calls on each device (zero when the library is loaded), and
// behind it what take_word_kernel last took out of it.
static __device__ unsigned int g_packed_err[4];

// One step on the device: kernels of other streams may be setting bits meanwhile, and a bit set
// between a copy and a memset would be cleared unseen.
static __global__ void take_word_kernel() { g_packed_err[1] = atomicExch(&g_packed_err[0], 0u); }

namespace fa {
namespace {

std::mutex g_mu;
unsigned int* g_err_ptr[kMaxDevices] = {};

// Longest packed axis and longest request: positions, tile numbers and windows stay far from
// the ends of 32 bits.
constexpr int kMaxTokens = 1 << 28;
constexpr int kMaxTreeWords = 1024;  // 64 new tokens of a request each

int bad(const char* arg, const std::string& reason) { return set_error(FA_ERR_INVALID_ARG, arg, reason.c_str()); }
int cuda_bad(const char* where, cudaError_t e) { return set_error(FA_ERR_CUDA, where, cudaGetErrorString(e)); }

// Device address of the error word.  The look-up may load the library's code on the device, so
// it runs with relaxed capture checks: a first call inside a graph capture is fine.
int err_word(unsigned int** out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_bad("cudaGetDevice", e);
    if (dev < 0 || dev >= kMaxDevices) return set_error(FA_ERR_UNSUPPORTED, "device", "device index too large");
    // a thread's first call (an autograd worker's, say) makes tensor maps before it launches
    // anything: the driver refuses that until the device's context is current in the thread
    if ((e = cudaSetDevice(dev)) != cudaSuccess) return cuda_bad("cudaSetDevice", e);
    std::lock_guard<std::mutex> lk(g_mu);
    if (g_err_ptr[dev] == nullptr) {
        cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
        cudaThreadExchangeStreamCaptureMode(&mode);
        void* p = nullptr;
        e = cudaGetSymbolAddress(&p, g_packed_err);
        cudaThreadExchangeStreamCaptureMode(&mode);
        if (e != cudaSuccess || p == nullptr) return cuda_bad("cudaGetSymbolAddress", e);
        g_err_ptr[dev] = static_cast<unsigned int*>(p);
    }
    *out = g_err_ptr[dev];
    return FA_OK;
}

int check_count(const char* name, long long v, long long lo, long long hi) {
    if (v < lo || v > hi)
        return bad(name, "must be in [" + std::to_string(lo) + ", " + std::to_string(hi) + "], got " + std::to_string(v));
    return FA_OK;
}

int check_ptr(const void* p, const char* name, size_t align) {
    if (p == nullptr) return bad(name, "null pointer");
    if (reinterpret_cast<uintptr_t>(p) % align != 0) return bad(name, "must be " + std::to_string(align) + "-byte aligned");
    return FA_OK;
}

// Common checks of a call's heads, types and mask.
int check_common(int N, int H, int H_kv, int d, float scale, int causal, int window, int fill, int dtype) {
    int rc;
    if ((rc = check_count("N", N, 1, kMaxTokens))) return rc;
    if ((rc = check_count("H", H, 1, 65536))) return rc;
    if ((rc = check_count("H_kv", H_kv, 1, 65536))) return rc;
    if (H % H_kv != 0)
        return bad("H_kv", "num_kv_heads " + std::to_string(H_kv) + " must divide num_heads " + std::to_string(H));
    if (dtype != FA_F32 && dtype != FA_F16 && dtype != FA_BF16)
        return bad("dtype", "unsupported dtype " + std::to_string(dtype) + " (expected FA_F32, FA_F16 or FA_BF16)");
    if (d <= 0) return bad("d", "must be > 0, got " + std::to_string(d));
    if (!head_dim_supported(d))
        return set_error(FA_ERR_UNSUPPORTED, "d",
                         ("head dim " + std::to_string(d) + " not supported (32, 64, 96, 128 or 256)").c_str());
    if (!(isfinite(scale) && scale > 0.f)) return bad("scale", "must be finite and > 0");
    if (causal != 0 && causal != 1) return bad("causal", "must be 0 or 1");
    if (window < 0) return bad("window_size", "must be >= 0 (0 = no window)");
    if (fill != 0 && fill != 1) return bad("fill", "must be 0 or 1");
    return FA_OK;
}

int elem_bytes(int dtype) { return dtype == FA_F32 ? 4 : 2; }

// Element strides `s` (n of them): positive, whole 16-byte pieces.  Entries [q8_first, q8_last) are
// those of an 8-bit cache.
int check_strides(const long long* s, int n, int dtype, int q8_first = 0, int q8_last = 0) {
    for (int i = 0; i < n; ++i) {
        const int es = i >= q8_first && i < q8_last ? 1 : elem_bytes(dtype);
        if (s[i] <= 0 || s[i] >= (1ll << 38) || s[i] * es % 16 != 0)
            return bad("strides", "entry " + std::to_string(i) + " (" + std::to_string(s[i]) +
                                      ") must be > 0 and a multiple of 16 bytes");
    }
    return FA_OK;
}

// A call's outputs may overlap none of its inputs: blocks read and write at no set time.
struct Span {
    const char* name;
    const void* p;
    long long bytes;
};
template <int kIn, int kOut>
int check_apart(const Span (&in)[kIn], const Span (&out)[kOut]) {
    for (const Span& o : out)
        for (const Span& i : in) {
            const uintptr_t op = reinterpret_cast<uintptr_t>(o.p), ip = reinterpret_cast<uintptr_t>(i.p);
            if (op < ip + i.bytes && ip < op + o.bytes)
                return bad(o.name, std::string("must not overlap ") + i.name);
        }
    return FA_OK;
}

// Whether the tensor-core kernel's TMA boxes can address the call.
bool use_tensor_cores(const PackedFwd& a) {
    if (a.dtype == FA_F32 || a.H / a.H_kv > 128) return false;
    if (!a.paged() || a.q8()) return true;
    const int bn = a.d == 256 ? 64 : 128;  // keys per tile
    // pages of whole 8-row swizzle atoms that divide a tile, or are made of whole tiles
    return a.page_size % 8 == 0 && (bn % a.page_size == 0 || a.page_size % bn == 0);
}

bool bwd_tensor_cores(const PackedBwd& a) { return a.dtype != FA_F32; }

size_t fwd_bytes(const PackedFwd& a) {
    size_t n = 0;
    if (use_tensor_cores(a))
        launch_packed_fwd(a, nullptr, &n, nullptr);
    else
        launch_packed_fwd_simt(a, nullptr, &n, nullptr);
    return n;
}

int run_fwd(PackedFwd& a, void* ws, size_t ws_bytes, cudaStream_t st) {
    int rc;
    if ((rc = err_word(&a.err))) return rc;
    if (a.window > kOpen) a.window = kOpen;  // wider than any sequence: the same mask
    const size_t need = fwd_bytes(a);
    if (ws == nullptr || ws_bytes < need)
        return bad("workspace", "needs " + std::to_string(need) + " bytes, got " + std::to_string(ws ? ws_bytes : 0));
    if ((rc = check_ptr(ws, "workspace", 256))) return rc;
    size_t n = 0;
    const cudaError_t e = use_tensor_cores(a) ? launch_packed_fwd(a, ws, &n, st) : launch_packed_fwd_simt(a, ws, &n, st);
    if (e != cudaSuccess) return cuda_bad("forward launch", e);
    return FA_OK;
}

}  // namespace

int sm_count() {
    static std::atomic<int> sms[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
    int n = sms[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
        sms[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

unsigned long long next_tag() {
    static std::atomic<unsigned long long> last{(unsigned long long)time(nullptr) << 20};
    unsigned long long t;
    do t = (last.fetch_add(1, std::memory_order_relaxed) + 1) & ((1ull << 48) - 1);
    while (t == 0);
    return t;
}

int packed_take_error_word(unsigned int* word) {
    *word = 0;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_bad("cudaGetDevice", e);
    if (dev < 0 || dev >= kMaxDevices) return FA_OK;
    std::lock_guard<std::mutex> lk(g_mu);
    if (g_err_ptr[dev] == nullptr) return FA_OK;  // no such call on this device yet
    e = cudaMemcpy(word, g_err_ptr[dev], sizeof(unsigned int), cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_bad("cudaMemcpy", e);
    if (*word != 0) {
        take_word_kernel<<<1, 1>>>();  // on the stream of the copies
        if ((e = cudaGetLastError()) != cudaSuccess) return cuda_bad("take_word launch", e);
        e = cudaMemcpy(word, g_err_ptr[dev] + 1, sizeof(unsigned int), cudaMemcpyDeviceToHost);
        if (e != cudaSuccess) return cuda_bad("cudaMemcpy", e);
    }
    return FA_OK;
}

}  // namespace fa

using namespace fa;

extern "C" {

size_t fa_varlen_workspace_bytes(int N, int T_q, int T_k, int H, int H_kv, int d, int dtype, int backward) {
    if (check_common(N, H, H_kv, d, 1.f, 0, 0, 0, dtype) != FA_OK || T_q < 0 || T_k < 0) return 0;
    if (backward) {
        PackedBwd b = {};
        b.N = N, b.T_q = T_q, b.T_k = T_k, b.H = H, b.H_kv = H_kv, b.d = d, b.dtype = dtype, b.deterministic = 1;
        return bwd_plan_layout(b, bwd_tensor_cores(b), nullptr, nullptr);
    }
    PackedFwd a = {};
    static const int some = 0;
    a.cu_k = &some;  // packed
    a.N = N, a.T_q = T_q, a.T_k = T_k, a.H = H, a.H_kv = H_kv, a.d = d, a.dtype = dtype;
    return fwd_bytes(a);
}

size_t fa_paged_workspace_bytes_ex(int N, int T_q, int H, int H_kv, int d, int page_size, int max_pages, int dtype,
                                   int quantised) {
    if (check_common(N, H, H_kv, d, 1.f, 0, 0, 0, dtype) != FA_OK || T_q < 0 || page_size <= 0 || max_pages <= 0) return 0;
    PackedFwd a = {};
    static const uint8_t some = 0;
    if (quantised) a.k_exp = a.v_exp = &some;
    a.N = N, a.T_q = T_q, a.H = H, a.H_kv = H_kv, a.d = d, a.dtype = dtype, a.page_size = page_size;
    a.max_pages = max_pages;
    return fwd_bytes(a);
}

size_t fa_paged_workspace_bytes(int N, int T_q, int H, int H_kv, int d, int page_size, int dtype) {
    return fa_paged_workspace_bytes_ex(N, T_q, H, H_kv, d, page_size, 1, dtype, 0);
}

int fa_varlen_fwd(const void* Q, const void* K, const void* V, void* O, float* LSE, const int* cu_q, const int* cu_k,
                  int N, int T_q, int T_k, int H, int H_kv, int d, const long long* strides, float scale, int causal,
                  int window_size, int fill, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
    clear_error();
    int rc;
    if ((rc = check_common(N, H, H_kv, d, scale, causal, window_size, fill, dtype))) return rc;
    if ((rc = check_count("T_q", T_q, 0, kMaxTokens)) || (rc = check_count("T_k", T_k, 0, kMaxTokens))) return rc;
    if ((rc = check_ptr(cu_q, "cu_q", 4)) || (rc = check_ptr(cu_k, "cu_k", 4))) return rc;
    if (T_q == 0) return FA_OK;  // no rows to write
    if ((rc = check_ptr(Q, "Q", 16)) || (rc = check_ptr(O, "O", 16)) || (rc = check_ptr(LSE, "LSE", 4))) return rc;
    if (T_k > 0 && ((rc = check_ptr(K, "K", 16)) || (rc = check_ptr(V, "V", 16)))) return rc;
    const long long dense[8] = {(long long)H * d, d, (long long)H_kv * d, d, (long long)H_kv * d, d, (long long)H * d, d};
    const long long* s = strides ? strides : dense;
    if ((rc = check_strides(s, 8, dtype))) return rc;
    PackedFwd a = {};
    a.Q = Q, a.K = K, a.V = V, a.O = O, a.LSE = LSE, a.cu_q = cu_q, a.cu_k = cu_k;
    a.N = N, a.T_q = T_q, a.T_k = T_k, a.H = H, a.H_kv = H_kv, a.d = d;
    a.q = {s[0], s[1]}, a.k = {s[2], s[3]}, a.v = {s[4], s[5]}, a.o = {s[6], s[7]};
    a.scale = scale, a.causal = causal, a.window = window_size, a.fill = fill, a.dtype = dtype;
    return run_fwd(a, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

int fa_varlen_bwd(const void* dO, const void* Q, const void* K, const void* V, const void* O, const float* LSE, void* dQ,
                  void* dK, void* dV, const int* cu_q, const int* cu_k, int N, int T_q, int T_k, int H, int H_kv, int d,
                  const long long* strides, float scale, int causal, int window_size, int deterministic, int fill,
                  int dtype, void* workspace, size_t workspace_bytes, void* stream) {
    clear_error();
    int rc;
    if ((rc = check_common(N, H, H_kv, d, scale, causal, window_size, fill, dtype))) return rc;
    if (deterministic != 0 && deterministic != 1) return bad("deterministic", "must be 0 or 1");
    if ((rc = check_count("T_q", T_q, 0, kMaxTokens)) || (rc = check_count("T_k", T_k, 0, kMaxTokens))) return rc;
    if ((rc = check_ptr(cu_q, "cu_q", 4)) || (rc = check_ptr(cu_k, "cu_k", 4))) return rc;
    if (T_q == 0 && T_k == 0) return FA_OK;
    if (T_q > 0 && ((rc = check_ptr(dO, "dO", 16)) || (rc = check_ptr(Q, "Q", 16)) || (rc = check_ptr(O, "O", 16)) ||
                    (rc = check_ptr(LSE, "LSE", 4)) || (rc = check_ptr(dQ, "dQ", 16))))
        return rc;
    if (T_k > 0 && ((rc = check_ptr(K, "K", 16)) || (rc = check_ptr(V, "V", 16)) || (rc = check_ptr(dK, "dK", 16)) ||
                    (rc = check_ptr(dV, "dV", 16))))
        return rc;
    const long long qr = (long long)H * d, kr = (long long)H_kv * d;
    const long long dense[16] = {qr, d, qr, d, kr, d, kr, d, qr, d, qr, d, kr, d, kr, d};
    const long long* s = strides ? strides : dense;
    if ((rc = check_strides(s, 16, dtype))) return rc;
    PackedBwd a = {};
    a.dO = dO, a.Q = Q, a.K = K, a.V = V, a.O = O, a.LSE = LSE, a.dQ = dQ, a.dK = dK, a.dV = dV;
    a.cu_q = cu_q, a.cu_k = cu_k, a.N = N, a.T_q = T_q, a.T_k = T_k, a.H = H, a.H_kv = H_kv, a.d = d;
    a.sdo = {s[0], s[1]}, a.sq = {s[2], s[3]}, a.sk = {s[4], s[5]}, a.sv = {s[6], s[7]}, a.so = {s[8], s[9]};
    a.sdq = {s[10], s[11]}, a.sdk = {s[12], s[13]}, a.sdv = {s[14], s[15]};
    a.scale = scale, a.causal = causal, a.window = window_size > kOpen ? kOpen : window_size;
    a.deterministic = deterministic, a.fill = fill, a.dtype = dtype;
    if ((rc = err_word(&a.err))) return rc;
    const bool tc = bwd_tensor_cores(a);
    BwdPlan p;
    const size_t need = bwd_plan_layout(a, tc, workspace, &p);
    if (workspace == nullptr || workspace_bytes < need)
        return bad("workspace", "needs " + std::to_string(need) + " bytes, got " +
                                    std::to_string(workspace ? workspace_bytes : 0));
    if ((rc = check_ptr(workspace, "workspace", 256))) return rc;
    // the largest grid is one CTA per 16 rows of a query tile or per piece of a key tile and head
    if ((double)p.max_units * 8 > 1.0e9 || (double)p.max_work * H_kv * 4 > 1.0e9 || H > 65535)
        return bad("shape", "tensor too large");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = launch_bwd_plan(a, p, tc, st);
    if (e != cudaSuccess) return cuda_bad("plan launch", e);
    if ((e = launch_packed_preprocess(a, p, st)) != cudaSuccess) return cuda_bad("preprocess launch", e);
    e = !tc ? launch_packed_bwd_simt(a, p, st) : d == 256 ? launch_packed_bwd_d256(a, p, st) : launch_packed_bwd(a, p, st);
    if (e == cudaSuccess && deterministic && (!tc || d == 256)) e = launch_packed_dq_ordered(a, p, st);
    if (e != cudaSuccess) return cuda_bad("main kernel launch", e);
    if ((e = launch_packed_dq(a, p, st)) != cudaSuccess) return cuda_bad("dq launch", e);
    return FA_OK;
}

int fa_paged_fwd_ex(const void* Q, const void* K_cache, const void* V_cache, const void* K_exp, const void* V_exp, void* O,
                    float* LSE, const int* block_table, const int* cu_q, const int* seq_lens, const long long* tree,
                    int tree_words, int N, int T_q, int num_pages, int page_size, int max_pages, int H, int H_kv, int d,
                    const long long* strides, float scale, int causal, int window_size, int fill, int dtype,
                    void* workspace, size_t workspace_bytes, void* stream) {
    clear_error();
    int rc;
    if ((rc = check_common(N, H, H_kv, d, scale, causal, window_size, fill, dtype))) return rc;
    if ((rc = check_count("T_q", T_q, 0, kMaxTokens)) || (rc = check_count("num_pages", num_pages, 1, kMaxTokens)) ||
        (rc = check_count("page_size", page_size, 1, kMaxTokens)) ||
        (rc = check_count("max_pages", max_pages, 1, kMaxTokens)))
        return rc;
    if ((K_exp == nullptr) != (V_exp == nullptr))
        return bad(K_exp ? "V_exp" : "K_exp", "an 8-bit cache has exponents for both K and V");
    if (tree != nullptr) {
        if (causal != 1) return bad("causal", "must be 1 with a tree");
        if (window_size != 0) return bad("window_size", "must be 0 with a tree");
        if ((rc = check_count("tree_words", tree_words, 1, kMaxTreeWords)) || (rc = check_ptr(tree, "tree", 8))) return rc;
    }
    if ((rc = check_ptr(block_table, "block_table", 4)) || (rc = check_ptr(cu_q, "cu_q", 4)) ||
        (rc = check_ptr(seq_lens, "seq_lens", 4)))
        return rc;
    if (T_q == 0) return FA_OK;
    if ((rc = check_ptr(Q, "Q", 16)) || (rc = check_ptr(K_cache, "K_cache", 16)) ||
        (rc = check_ptr(V_cache, "V_cache", 16)) || (rc = check_ptr(O, "O", 16)) || (rc = check_ptr(LSE, "LSE", 4)))
        return rc;
    if (K_exp && ((rc = check_ptr(K_exp, "K_exp", 16)) || (rc = check_ptr(V_exp, "V_exp", 16)))) return rc;
    const long long kr = (long long)H_kv * d, qr = (long long)H * d;
    const long long dense[10] = {qr, d, kr * page_size, kr, d, kr * page_size, kr, d, qr, d};
    const long long* s = strides ? strides : dense;
    if ((rc = check_strides(s, 10, dtype, 2, K_exp ? 8 : 2))) return rc;
    PackedFwd a = {};
    a.Q = Q, a.K = K_cache, a.V = V_cache, a.O = O, a.LSE = LSE;
    a.k_exp = static_cast<const uint8_t*>(K_exp), a.v_exp = static_cast<const uint8_t*>(V_exp);
    a.tree = reinterpret_cast<const unsigned long long*>(tree), a.tree_words = tree ? tree_words : 0;
    a.cu_q = cu_q, a.seq_lens = seq_lens, a.table = block_table;
    a.N = N, a.T_q = T_q, a.H = H, a.H_kv = H_kv, a.d = d;
    a.pages = num_pages, a.page_size = page_size, a.max_pages = max_pages;
    a.q = {s[0], s[1]}, a.k_page = s[2], a.k = {s[3], s[4]}, a.v_page = s[5], a.v = {s[6], s[7]}, a.o = {s[8], s[9]};
    a.scale = scale, a.causal = causal, a.window = window_size, a.fill = fill, a.dtype = dtype;
    return run_fwd(a, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

int fa_paged_fwd(const void* Q, const void* K_cache, const void* V_cache, void* O, float* LSE, const int* block_table,
                 const int* cu_q, const int* seq_lens, int N, int T_q, int num_pages, int page_size, int max_pages, int H,
                 int H_kv, int d, const long long* strides, float scale, int causal, int window_size, int fill, int dtype,
                 void* workspace, size_t workspace_bytes, void* stream) {
    return fa_paged_fwd_ex(Q, K_cache, V_cache, nullptr, nullptr, O, LSE, block_table, cu_q, seq_lens, nullptr, 0, N, T_q,
                           num_pages, page_size, max_pages, H, H_kv, d, strides, scale, causal, window_size, fill, dtype,
                           workspace, workspace_bytes, stream);
}

int fa_page_slots(const int* ctx_lens, const int* cu_q, const int* free_pages, const int* free_start, int* block_table,
                  long long* slots, int* positions, int* seq_lens, int* free_next, int N, int T, int num_free,
                  int page_size, int max_pages, void* stream) {
    clear_error();
    int rc;
    if ((rc = check_count("N", N, 1, kMaxTokens)) || (rc = check_count("T", T, 0, kMaxTokens)) ||
        (rc = check_count("num_free", num_free, 0, kMaxTokens)) ||
        (rc = check_count("page_size", page_size, 1, kMaxTokens)) ||
        (rc = check_count("max_pages", max_pages, 1, kMaxTokens)))
        return rc;
    if ((rc = check_ptr(ctx_lens, "ctx_lens", 4)) || (rc = check_ptr(cu_q, "cu_q", 4)) ||
        (rc = check_ptr(free_start, "free_start", 4)) || (rc = check_ptr(block_table, "block_table", 4)) ||
        (rc = check_ptr(seq_lens, "seq_lens", 4)) || (rc = check_ptr(free_next, "free_next", 4)))
        return rc;
    if (num_free > 0 && (rc = check_ptr(free_pages, "free_pages", 4))) return rc;
    if (T > 0 && ((rc = check_ptr(slots, "slots", 8)) || (rc = check_ptr(positions, "positions", 4)))) return rc;
    const Span in[] = {{"ctx_lens", ctx_lens, 4ll * N}, {"cu_q", cu_q, 4ll * (N + 1)},
                       {"free_pages", free_pages, 4ll * num_free}, {"free_start", free_start, 4}};
    const Span out[] = {{"slots", slots, 8ll * T}, {"positions", positions, 4ll * T}, {"seq_lens", seq_lens, 4ll * N},
                        {"free_next", free_next, 4}, {"block_table", block_table, 4ll * N * max_pages}};
    if ((rc = check_apart(in, out))) return rc;
    PageSlots a = {};
    a.ctx_lens = ctx_lens, a.cu_q = cu_q, a.free_pages = free_pages, a.free_start = free_start;
    a.table = block_table, a.slots = slots, a.positions = positions, a.seq_lens = seq_lens, a.free_next = free_next;
    a.N = N, a.T = T, a.n_free = num_free, a.page_size = page_size, a.max_pages = max_pages;
    if ((rc = err_word(&a.err))) return rc;
    const cudaError_t e = launch_page_slots(a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_bad("page_slots launch", e);
    return FA_OK;
}

int fa_paged_write(const void* K, const void* V, const long long* slots, void* K_cache, void* V_cache, int T,
                   int num_pages, int page_size, int H_kv, int d, const long long* strides, int dtype, void* stream) {
    clear_error();
    int rc;
    if ((rc = check_common(1, H_kv, H_kv, d, 1.f, 0, 0, 0, dtype))) return rc;
    if ((rc = check_count("T", T, 0, kMaxTokens)) || (rc = check_count("num_pages", num_pages, 1, kMaxTokens)) ||
        (rc = check_count("page_size", page_size, 1, kMaxTokens)))
        return rc;
    if (T == 0) return FA_OK;
    if ((rc = check_ptr(K, "K", 16)) || (rc = check_ptr(V, "V", 16)) || (rc = check_ptr(slots, "slots", 8)) ||
        (rc = check_ptr(K_cache, "K_cache", 16)) || (rc = check_ptr(V_cache, "V_cache", 16)))
        return rc;
    const long long kr = (long long)H_kv * d;
    const long long dense[10] = {kr, d, kr, d, kr * page_size, kr, d, kr * page_size, kr, d};
    const long long* s = strides ? strides : dense;
    if ((rc = check_strides(s, 10, dtype))) return rc;
    const long long es = dtype == FA_F32 ? 4 : 2;
    PagedWrite a = {};
    a.K = K, a.V = V, a.K_cache = K_cache, a.V_cache = V_cache, a.slots = slots;
    a.T = T, a.H_kv = H_kv, a.cpr = (int)(d * es / 16), a.pages = num_pages, a.page_size = page_size;
    a.k = {s[0] * es, s[1] * es}, a.v = {s[2] * es, s[3] * es};
    a.kc_page = s[4] * es, a.kc = {s[5] * es, s[6] * es}, a.vc_page = s[7] * es, a.vc = {s[8] * es, s[9] * es};
    if ((rc = err_word(&a.err))) return rc;
    const cudaError_t e = launch_paged_write(a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_bad("paged_write launch", e);
    return FA_OK;
}

// The arguments that writing an 8-bit cache and reading it back share.
static int q8_args(PagedQ8& a, const void* K, const void* V, const void* K_cache, const void* V_cache, const void* K_exp,
                   const void* V_exp, const long long* slots, int T, int num_pages, int page_size, int H_kv, int d,
                   const long long* strides, int dtype) {
    int rc;
    if ((rc = check_common(1, H_kv, H_kv, d, 1.f, 0, 0, 0, dtype))) return rc;
    if ((rc = check_count("T", T, 0, kMaxTokens)) || (rc = check_count("num_pages", num_pages, 1, kMaxTokens)) ||
        (rc = check_count("page_size", page_size, 1, kMaxTokens)))
        return rc;
    if (T == 0) return FA_OK;
    if ((rc = check_ptr(K, "K", 16)) || (rc = check_ptr(V, "V", 16)) || (rc = check_ptr(slots, "slots", 8)) ||
        (rc = check_ptr(K_cache, "K_cache", 16)) || (rc = check_ptr(V_cache, "V_cache", 16)) ||
        (rc = check_ptr(K_exp, "K_exp", 16)) || (rc = check_ptr(V_exp, "V_exp", 16)))
        return rc;
    const long long kr = (long long)H_kv * d;
    const long long dense[10] = {kr, d, kr, d, kr * page_size, kr, d, kr * page_size, kr, d};
    const long long* s = strides ? strides : dense;
    if ((rc = check_strides(s, 10, dtype, 4, 10))) return rc;
    const long long es = elem_bytes(dtype);
    a.K = const_cast<void*>(K), a.V = const_cast<void*>(V);
    a.K_cache = const_cast<void*>(K_cache), a.V_cache = const_cast<void*>(V_cache), a.slots = slots;
    a.k_exp = static_cast<uint8_t*>(const_cast<void*>(K_exp)), a.v_exp = static_cast<uint8_t*>(const_cast<void*>(V_exp));
    a.T = T, a.H_kv = H_kv, a.d = d, a.pages = num_pages, a.page_size = page_size, a.dtype = dtype;
    a.k = {s[0] * es, s[1] * es}, a.v = {s[2] * es, s[3] * es};
    a.kc_page = s[4], a.kc = {s[5], s[6]}, a.vc_page = s[7], a.vc = {s[8], s[9]};
    return err_word(&a.err);
}

int fa_paged_write_q8(const void* K, const void* V, const long long* slots, void* K_cache, void* V_cache, void* K_exp,
                      void* V_exp, int T, int num_pages, int page_size, int H_kv, int d, const long long* strides,
                      int dtype, void* stream) {
    clear_error();
    PagedQ8 a = {};
    const int rc = q8_args(a, K, V, K_cache, V_cache, K_exp, V_exp, slots, T, num_pages, page_size, H_kv, d, strides, dtype);
    if (rc != FA_OK || T == 0) return rc;
    const cudaError_t e = launch_paged_write_q8(a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_bad("paged_write_q8 launch", e);
    return FA_OK;
}

int fa_paged_read_q8(const void* K_cache, const void* V_cache, const void* K_exp, const void* V_exp, const long long* slots,
                     void* K, void* V, int T, int num_pages, int page_size, int H_kv, int d, const long long* strides,
                     int dtype, void* stream) {
    clear_error();
    PagedQ8 a = {};
    const int rc = q8_args(a, K, V, K_cache, V_cache, K_exp, V_exp, slots, T, num_pages, page_size, H_kv, d, strides, dtype);
    if (rc != FA_OK || T == 0) return rc;
    const cudaError_t e = launch_paged_read_q8(a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_bad("paged_read_q8 launch", e);
    return FA_OK;
}

int fa_tree_mask(const int* parents, const int* cu_q, const int* ctx_lens, long long* tree, int* positions, int N, int T,
                 int words, void* stream) {
    clear_error();
    int rc;
    if ((rc = check_count("N", N, 1, kMaxTokens)) || (rc = check_count("T", T, 0, kMaxTokens)) ||
        (rc = check_count("words", words, 1, kMaxTreeWords)))
        return rc;
    if ((rc = check_ptr(cu_q, "cu_q", 4)) || (rc = check_ptr(ctx_lens, "ctx_lens", 4))) return rc;
    if (T == 0) return FA_OK;
    if ((rc = check_ptr(parents, "parents", 4)) || (rc = check_ptr(tree, "tree", 8)) ||
        (rc = check_ptr(positions, "positions", 4)))
        return rc;
    const Span in[] = {{"parents", parents, 4ll * T}, {"cu_q", cu_q, 4ll * (N + 1)}, {"ctx_lens", ctx_lens, 4ll * N}};
    const Span out[] = {{"tree", tree, 8ll * T * words}, {"positions", positions, 4ll * T}};
    if ((rc = check_apart(in, out))) return rc;
    TreeMask a = {};
    a.parents = parents, a.cu_q = cu_q, a.ctx_lens = ctx_lens;
    a.tree = reinterpret_cast<unsigned long long*>(tree), a.positions = positions;
    a.N = N, a.T = T, a.words = words;
    if ((rc = err_word(&a.err))) return rc;
    const cudaError_t e = launch_tree_mask(a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_bad("tree_mask launch", e);
    return FA_OK;
}

int fa_paged_keep(const int* path, const int* count, const int* cu_q, const int* seq_lens, const int* block_table,
                  void* const* K_caches, void* const* V_caches, void* const* K_exps, void* const* V_exps, int layers,
                  int N, int T, int num_pages, int page_size, int max_pages, int H_kv, int d, const long long* strides,
                  int dtype, void* stream) {
    clear_error();
    int rc;
    if ((rc = check_common(N, H_kv, H_kv, d, 1.f, 0, 0, 0, dtype))) return rc;
    if ((rc = check_count("T", T, 0, kMaxTokens)) || (rc = check_count("layers", layers, 1, 65536)) ||
        (rc = check_count("num_pages", num_pages, 1, kMaxTokens)) ||
        (rc = check_count("page_size", page_size, 1, kMaxTokens)) ||
        (rc = check_count("max_pages", max_pages, 1, kMaxTokens)))
        return rc;
    if ((rc = check_ptr(count, "count", 4)) || (rc = check_ptr(cu_q, "cu_q", 4)) ||
        (rc = check_ptr(seq_lens, "seq_lens", 4)) || (rc = check_ptr(block_table, "block_table", 4)) ||
        (rc = check_ptr(K_caches, "K_caches", 8)) || (rc = check_ptr(V_caches, "V_caches", 8)))
        return rc;
    if ((K_exps == nullptr) != (V_exps == nullptr))
        return bad(K_exps ? "V_exps" : "K_exps", "an 8-bit cache has exponents for both K and V");
    if (T == 0) return FA_OK;
    if ((rc = check_ptr(path, "path", 4))) return rc;
    for (int i = 0; i < layers; ++i)
        if ((rc = check_ptr(K_caches[i], "K_caches", 16)) || (rc = check_ptr(V_caches[i], "V_caches", 16)) ||
            (K_exps && ((rc = check_ptr(K_exps[i], "K_exps", 16)) || (rc = check_ptr(V_exps[i], "V_exps", 16)))))
            return rc;
    // a tensor given twice would be moved twice, by blocks that do not wait for one another
    std::vector<const void*> all;
    try {
        for (void* const* list : {K_caches, V_caches, K_exps, V_exps})
            if (list) all.insert(all.end(), list, list + layers);
    } catch (const std::bad_alloc&) {
        return set_error(FA_ERR_NOMEM, "layers", "out of host memory");
    }
    std::sort(all.begin(), all.end());
    if (std::adjacent_find(all.begin(), all.end()) != all.end()) return bad("K_caches", "the same tensor is given twice");
    const long long kr = (long long)H_kv * d;
    const long long dense[6] = {kr * page_size, kr, d, kr * page_size, kr, d};
    const long long* s = strides ? strides : dense;
    if ((rc = check_strides(s, 6, dtype, 0, K_exps ? 6 : 0))) return rc;
    const long long es = K_exps ? 1 : elem_bytes(dtype);
    PagedKeep a = {};
    a.path = path, a.count = count, a.cu_q = cu_q, a.seq_lens = seq_lens, a.table = block_table;
    a.N = N, a.T = T, a.H_kv = H_kv, a.cpr = (int)(d * es / 16);
    a.pages = num_pages, a.page_size = page_size, a.max_pages = max_pages;
    a.kc_page = s[0] * es, a.kc = {s[1] * es, s[2] * es}, a.vc_page = s[3] * es, a.vc = {s[4] * es, s[5] * es};
    if ((rc = err_word(&a.err))) return rc;
    for (int l0 = 0; l0 < layers; l0 += kKeepLayers) {
        a.layers = layers - l0 < kKeepLayers ? layers - l0 : kKeepLayers;
        for (int i = 0; i < a.layers; ++i) {
            a.K[i] = K_caches[l0 + i], a.V[i] = V_caches[l0 + i];
            a.k_exp[i] = K_exps ? static_cast<uint8_t*>(K_exps[l0 + i]) : nullptr;
            a.v_exp[i] = V_exps ? static_cast<uint8_t*>(V_exps[l0 + i]) : nullptr;
        }
        const cudaError_t e = launch_paged_keep(a, static_cast<cudaStream_t>(stream));
        if (e != cudaSuccess) return cuda_bad("paged_keep launch", e);
    }
    return FA_OK;
}

static int page_trim(PageTrim a, cudaStream_t st) {
    clear_error();
    int rc;
    if ((rc = check_count("N", a.N, 1, kMaxTokens)) || (rc = check_count("T", a.T, 0, kMaxTokens)) ||
        (rc = check_count("num_free", a.n_free, 0, kMaxTokens)) ||
        (rc = check_count("page_size", a.page_size, 1, kMaxTokens)) ||
        (rc = check_count("max_pages", a.max_pages, 1, kMaxTokens)))
        return rc;
    if ((rc = check_ptr(a.count, "count", 4)) || (rc = check_ptr(a.cu_q, "cu_q", 4)) ||
        (rc = check_ptr(a.seq_lens, "seq_lens", 4)) || (rc = check_ptr(a.table, "block_table", 4)) ||
        (rc = check_ptr(a.free_start, "free_start", 4)) || (rc = check_ptr(a.lens, "lens", 4)) ||
        (rc = check_ptr(a.free_next, "free_next", 4)))
        return rc;
    if (a.n_free > 0 && (rc = check_ptr(a.free_pages, "free_pages", 4))) return rc;
    if (a.T > 0 && (rc = check_ptr(a.path, "path", 4))) return rc;
    const Span in[] = {{"count", a.count, 4ll * a.N}, {"cu_q", a.cu_q, 4ll * (a.N + 1)}, {"seq_lens", a.seq_lens, 4ll * a.N},
                       {"block_table", a.table, 4ll * a.N * a.max_pages}, {"free_start", a.free_start, 4},
                       {"path", a.path, 4ll * a.T}};
    const Span out[] = {{"free_pages", a.free_pages, 4ll * a.n_free}, {"lens", a.lens, 4ll * a.N}, {"free_next", a.free_next, 4}};
    if ((rc = check_apart(in, out))) return rc;
    if ((rc = err_word(&a.err))) return rc;
    const cudaError_t e = launch_page_trim(a, st);
    if (e != cudaSuccess) return cuda_bad("page_trim launch", e);
    return FA_OK;
}

int fa_page_trim(const int* count, const int* cu_q, const int* seq_lens, const int* block_table, int* free_pages,
                 const int* free_start, int* lens, int* free_next, int N, int num_free, int page_size, int max_pages,
                 void* stream) {
    PageTrim a = {};
    a.count = count, a.cu_q = cu_q, a.seq_lens = seq_lens, a.table = block_table, a.free_start = free_start;
    a.free_pages = free_pages, a.lens = lens, a.free_next = free_next;
    a.N = N, a.n_free = num_free, a.page_size = page_size, a.max_pages = max_pages;
    return page_trim(a, static_cast<cudaStream_t>(stream));
}

int fa_page_trim_ex(const int* path, const int* count, const int* cu_q, const int* seq_lens, const int* block_table,
                    int* free_pages, const int* free_start, int* lens, int* free_next, int N, int T, int num_free,
                    int page_size, int max_pages, void* stream) {
    PageTrim a = {};
    a.by_path = true, a.path = path, a.T = T;
    a.count = count, a.cu_q = cu_q, a.seq_lens = seq_lens, a.table = block_table, a.free_start = free_start;
    a.free_pages = free_pages, a.lens = lens, a.free_next = free_next;
    a.N = N, a.n_free = num_free, a.page_size = page_size, a.max_pages = max_pages;
    return page_trim(a, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
